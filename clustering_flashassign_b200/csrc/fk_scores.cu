// Score kernels without a bias (one translation unit each, for the build's sake).
#include "fk_scores.cuh"

namespace fk {
namespace soft {

int launch_scores(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
      cudaStream_t s) {
  return scores_stats<false>(tx, tc, f, a, fmt, err, s);
}

}  // namespace soft
}  // namespace fk
