// Operand copies of the soft assignment products.
#include "fk_logprob.cuh"

namespace fk {
namespace soft {
namespace {

template <typename T>
__global__ void __launch_bounds__(256)
    k_operand(const T *src, long long rows, long long rows_per_b, int d, int dp, const float *bias, void *dst) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  copy_row<T>(src, r, rows_per_b, d, dp, bias && bias[r] == kNegInf, dst, lane);
}

template <typename T>
int launch_operand(const void *src, long long rows, long long rows_per_b, int d, int dp, const float *bias, void *dst, cudaStream_t s) {
  FK_CUDA(launch_pdl(k_operand<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const T *>(src), rows,
                     rows_per_b, d, dp, bias, dst));
  return launched();
}

}  // namespace

int operand(const void *src, int dtype, long long rows, long long rows_per_b, int d, int dp, const float *bias, void *dst, cudaStream_t s) {
  if (dtype == FK_F32) return launch_operand<float>(src, rows, rows_per_b, d, dp, bias, dst, s);
  return launch_operand<__half>(src, rows, rows_per_b, d, dp, bias, dst, s);  // 16-bit rows are copied as bits
}

}  // namespace soft
}  // namespace fk
