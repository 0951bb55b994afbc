// Forward entry points of the token log probabilities.
#include <mutex>
#include <set>

#include "fk_logprob.cuh"

namespace fk {
namespace soft {
namespace {

FwdSpace fwd_space(const Dims &m, int top, void *base) {
  FwdSpace f = {};
  f.p = plan_runs(m.B, m.N, m.K, m.d, m.pairs, m.planes, m.dp * 2 * m.planes);
  f.L = list_length(top);
  Carve w(base);
  const long long parts = f.parts = 3 * f.p.runs;
  f.part = (float4 *)w.take((size_t)m.B * m.N * parts * sizeof(float4));
  if (f.L) {
    f.top_v = (float *)w.take((size_t)m.B * m.N * parts * f.L * 4);
    f.top_i = (int32_t *)w.take((size_t)m.B * m.N * parts * f.L * 4);
    if (m.B * m.N > kJoinBlockRows) f.max_norm2 = (unsigned *)w.take((size_t)m.B * 4);
  }
  if (m.planes == 3) {
    f.xs = w.take((size_t)m.B * 3 * m.N * m.dp * 2);
    f.cs = w.take((size_t)m.B * 3 * m.K * m.dp * 2);
  }
  f.bytes = w.off;
  return f;
}

}  // namespace

int check_registers(const void *kernel, int regs) {
  static std::mutex mu;
  static std::set<const void *> good;
  std::lock_guard<std::mutex> lk(mu);
  if (good.count(kernel)) return FK_OK;
  cudaFuncAttributes at;
  FK_CUDA(cudaFuncGetAttributes(&at, kernel));
  if (at.numRegs != regs)
    return set_error(FK_ECUDA, "tile kernel built with " + std::to_string(at.numRegs) + " registers, not " +
                                   std::to_string(regs));
  good.insert(kernel);
  return FK_OK;
}

}  // namespace soft
}  // namespace fk

using namespace fk;
using namespace fk::soft;

extern "C" {

int fk_logprob_workspace(const fk_shape *shape, int top, long long *bytes) {
  FK_TRY(check_soft(shape, 1.f));
  if (!bytes) return set_error(FK_EINVAL, "bytes is NULL");
  if (top < 0 || top > kMaxTop || top > shape->K) return set_error(FK_EINVAL, "top must be in [0, min(K, 28)]");
  const FwdSpace f = fwd_space(dims_of(*shape), top, nullptr);
  if (too_many(f.p, shape->B)) return set_error(FK_EUNSUPPORTED, "too many tiles");
  *bytes = (long long)f.bytes;
  return FK_OK;
}

int fk_logprob(const fk_shape *shape, const void *x, const void *c, const float *bias, float scale, const int32_t *ids,
               float *logp, float *lse, float *lse_rest, float *entropy, int top, int32_t *top_ids, float *top_logp, void *workspace,
               long long workspace_bytes, fk_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FK_TRY(check_soft(shape, scale));
  long long need = 0;
  FK_TRY(fk_logprob_workspace(shape, top, &need));
  const Dims m = dims_of(*shape);
  FK_TRY(check_ptr(c, "c", m.dtype != FK_F32));
  if (m.N == 0) return FK_OK;
  FK_TRY(check_ptr(x, "x", m.dtype != FK_F32));
  FK_TRY(check_ptr(ids, "ids", false));
  FK_TRY(check_ptr(logp, "logp", false));
  FK_TRY(check_ptr(lse, "lse", false));
  if (top) {
    FK_TRY(check_ptr(top_ids, "top_ids", false));
    FK_TRY(check_ptr(top_logp, "top_logp", false));
  }
  FK_TRY(check_ptr(workspace, "workspace", true));
  if (workspace_bytes < need) return set_error(FK_EINVAL, "workspace is smaller than fk_logprob_workspace asks for");
  FK_TRY(check_dev(x, "x"));
  FK_TRY(check_dev(c, "c"));
  FK_TRY(check_dev_opt(bias, "bias"));
  FK_TRY(check_dev(ids, "ids"));
  FK_TRY(check_dev(logp, "logp"));
  FK_TRY(check_dev(lse, "lse"));
  FK_TRY(check_dev_opt(lse_rest, "lse_rest"));
  FK_TRY(check_dev_opt(entropy, "entropy"));
  if (top) {
    FK_TRY(check_dev(top_ids, "top_ids"));
    FK_TRY(check_dev(top_logp, "top_logp"));
  }
  FK_TRY(check_dev(workspace, "workspace"));
  int *err = nullptr;
  FK_TRY(soft_error_word(&err));
  const FwdSpace f = fwd_space(m, top, workspace);
  const void *xo = x, *co = c;
  if (m.planes == 3) {
    FK_TRY(operand(x, m.dtype, m.B * m.N, m.N, m.d, m.dp, nullptr, f.xs, s));
    FK_TRY(operand(c, m.dtype, (long long)m.B * m.K, m.K, m.d, m.dp, nullptr, f.cs, s));
    xo = f.xs, co = f.cs;
  }
  const bool bf = m.dtype != FK_F16;
  CUtensorMap tx, tc;
  FK_TRY(map_16(&tx, xo, bf, m.dp, m.N, (long long)m.B * m.planes, m.dp, m.N * m.dp, tile::kK, tile::kRows));
  FK_TRY(map_16(&tc, co, bf, m.dp, m.K, (long long)m.B * m.planes, m.dp, (long long)m.K * m.dp, tile::kK,
                tile::kCols / f.p.cg));
  StatArgs a = {};
  a.scale2 = scale * kLog2e;
  a.bias = bias;
  a.ids = ids;
  a.N = m.N, a.K = m.K;
  a.parts = f.parts;
  a.L = f.L;
  a.part = f.part, a.top_v = f.top_v, a.top_i = f.top_i;
  FK_TRY((bias ? launch_scores_bias : launch_scores)(tx, tc, f, a, bf ? 1 : 0, err, s));
  JoinArgs j = {};
  j.part = f.part, j.top_v = f.top_v, j.top_i = f.top_i;
  j.ids = ids, j.x = x, j.c = c, j.bias = bias, j.scale = scale, j.unit2 = bias ? 1.f : scale * kLog2e;
  j.rows = m.B * m.N, j.N = m.N, j.K = m.K, j.d = m.d;
  j.parts = a.parts, j.L = f.L, j.cands = top ? std::min(m.K, top + kSpare) : 0, j.top = top;
  j.logp = logp, j.lse = lse, j.lse_rest = lse_rest, j.entropy = entropy, j.top_logp = top_logp, j.top_ids = top_ids;
  j.err = err;
  j.max_norm2 = f.max_norm2;
  j.vec = m.d * esize(m.dtype) % 16 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(c)) & 15) == 0;
  return launch_join(j, m.dtype, s);
}

}  // extern "C"
