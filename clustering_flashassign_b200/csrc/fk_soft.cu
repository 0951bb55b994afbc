// Shared state of the soft assignment operators: their device error word.
#include "fk_internal.h"

namespace fk {
namespace {
__device__ int g_soft_err;
}

int soft_error_word(int **out) {
  void *p = nullptr;
  FK_CUDA(cudaGetSymbolAddress(&p, g_soft_err));  // of the current device
  *out = static_cast<int *>(p);
  return FK_OK;
}

int read_soft_error(cudaStream_t s) {
  int *word = nullptr;
  FK_TRY(soft_error_word(&word));
  int h = DEV_OK;
  FK_CUDA(cudaMemcpyAsync(&h, word, sizeof(int), cudaMemcpyDeviceToHost, s));
  FK_CUDA(cudaStreamSynchronize(s));
  if (h == DEV_OK) return FK_OK;
  FK_CUDA(cudaMemsetAsync(word, 0, sizeof(int), s));
  FK_CUDA(cudaStreamSynchronize(s));
  if (h == DEV_TIMEOUT) return set_error(FK_ETIMEOUT, "a kernel's bounded wait expired");
  return set_error(FK_EINVAL, "a token id of K or more reached fk_logprob");
}

}  // namespace fk
