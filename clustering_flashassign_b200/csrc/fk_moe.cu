// A mixture-of-experts layer for a few tokens (the serving step): every token's
// best experts under a soft assignment to the router's rows, and their gated
// feed-forward layers, in two kernels.
//
//   s = x R^T,  p = softmax(s),  the k largest (lowest index on ties)
//   w_j = p_j / sum of the k chosen p   (renormalize), or p_j
//   h_j = act(x Wg_j^T) * (x Wu_j^T),   y = sum_j w_j h_j Wd_j^T
//
// With few tokens the layer is bound by reading the chosen experts' weights
// (3 F d values each) once from HBM; every expert is read for all its tokens
// together, as the sort-inverse update gathers the points of one cluster.
//
// k_route: one cluster of 8 CTAs per 8 tokens.  The CTAs share the experts;
// scores are summed in fp64 (products of 16-bit values are exact, so experts
// are ranked by their exact scores) and sent to the CTA of their token, which
// draws the k best.
//
// k_experts: a persistent kernel over units of weights, taken from a ticket
// counter in the order  gate/up of expert 0, 1, ..., down of expert 0, 1, ...
//   gate/up unit   8 gate rows and the 8 up rows of the same columns: the 16
//                  rows of one mma.sync m16n8k16, whose 8 columns are tokens,
//   down unit      16 rows of Wd against the expert's h.
// The 8 warps of a CTA split a unit's contraction, so that a unit is one round
// of loads deep, and join through shared memory.  A lane loads 16 consecutive
// bytes of a row; the contraction's order inside a 32-element step is free, so
// these 8 elements feed two MMA steps without a transpose.  (tcgen05 has
// nothing to offer here: 128 rows of weights would meet 8 token columns, and
// the weights would take a detour through shared memory; the register path
// streams them at the rate HBM gives.)
// A down unit waits until its expert's h is complete.  Tickets make that safe
// without a grid-wide barrier or a cooperative launch: whoever waits holds a
// later ticket than every unit it waits for, and those are held by CTAs that
// run already.  Products of the k experts are written per (token, slot) and
// the CTA that finishes a block of 16 output columns sums its slots in order,
// so results do not depend on the order of arrival.
//
// h is held as hi + lo of the weights' type (bf16: 16 significant bits; fp16:
// 22, of h / 64 to keep the type's range ahead of h), so that rounding it does
// not add to the result's own rounding.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fk_sm100.cuh"

namespace fk {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxTokens = 256;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;
constexpr int kRouteCtas = 8;  // CTAs of a cluster = tokens of a cluster
constexpr int kWarps = 8;
constexpr float kHalfScale = 1.f / 64.f;

struct MoeArgs {
  int T, E, d, F, k, act, renorm;
  const void *x, *router, *w_in, *w_out;
  void *y;
  int32_t *ids;
  float *weights;
  // workspace
  int *tickets;      // [0] next ticket, then per-expert finished gate/up units, then per-block finished down units
  void *hi, *lo;     // (T * k, F)
  float *part;       // (T * k, d)
  int *err;
  int counters;
};

template <typename T>
struct Two;
template <>
struct Two<__half> {
  static __device__ __forceinline__ float2 f(uint32_t v) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }
  static constexpr bool kBf = false;
};
template <>
struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ float2 f(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
  }
  static constexpr bool kBf = true;
};

// ------------------------------------------------------------------ routing
template <typename T>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(32 * kWarps) k_route(const MoeArgs a) {
  __shared__ double scores[kMaxExperts];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = (int)cluster.block_rank();
  const int t0 = (blockIdx.x / kRouteCtas) * kRouteCtas;
  const int nt = min(kRouteCtas, a.T - t0);
  pdl_wait();
  pdl_trigger();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.counters; i += gridDim.x * blockDim.x) a.tickets[i] = 0;
  const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + (size_t)t0 * a.d);
  const int n = a.d / 8;
  cluster.sync();  // every CTA of the cluster runs before its memory is written
  for (int e = cta * kWarps + warp; e < a.E; e += kRouteCtas * kWarps) {
    const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.router) + (size_t)e * a.d);
    double acc[kRouteCtas] = {};
    for (int i = lane; i < n; i += 32) {
      const uint4 rv = __ldg(r + i);
      const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
      double rd[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = Two<T>::f(rw[j]);
        rd[2 * j] = f.x;
        rd[2 * j + 1] = f.y;
      }
#pragma unroll
      for (int t = 0; t < kRouteCtas; ++t) {
        if (t < nt) {
          const uint4 xv = __ldg(x + (size_t)t * n + i);
          const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = Two<T>::f(xw[j]);
            acc[t] = fma((double)f.x, rd[2 * j], acc[t]);
            acc[t] = fma((double)f.y, rd[2 * j + 1], acc[t]);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kRouteCtas; ++t) {
      if (t < nt) {
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
        if (lane == 0) *cluster.map_shared_rank(scores + e, t) = acc[t];
      }
    }
  }
  cluster.sync();
  if (warp != 0 || cta >= nt) return;
  const int t = t0 + cta;
  constexpr int kPer = kMaxExperts / 32;
  const double none = -INFINITY;
  double v[kPer];
  double big = none;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane + 32 * j;
    v[j] = e < a.E ? scores[e] : none;
    nan |= !(v[j] == v[j]);
    if (v[j] > big) big = v[j];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) big = fmax(big, __shfl_xor_sync(0xffffffffu, big, o));
  nan = __any_sync(0xffffffffu, nan);
  float all = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (lane + 32 * j < a.E) all += expf((float)(v[j] - big));
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  uint32_t taken = 0;
  int my_e = 0;
  float my_p = 0.f, chosen = 0.f;
  for (int j = 0; j < a.k; ++j) {
    // the best expert left; NaN and -inf scores rank last, lowest index first
    double bv = none;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && !(taken >> i & 1u) && (be == 0x7fffffff || v[i] > bv)) {
        be = e;
        bv = v[i] > none ? v[i] : none;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double v2 = __shfl_xor_sync(0xffffffffu, bv, o);
      const int e2 = __shfl_xor_sync(0xffffffffu, be, o);
      if (v2 > bv || (v2 == bv && e2 < be)) {
        bv = v2;
        be = e2;
      }
    }
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    const float p = nan ? NAN : expf((float)(bv - big));
    chosen += p;
    if (lane == j) {
      my_e = be;
      my_p = p;
    }
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_e;
    a.weights[t * a.k + lane] = my_p / (a.renorm ? chosen : all);
  }
}

// ------------------------------------------------------------------ experts
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 stream16(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// h and the partial results are written by other CTAs of this kernel
__device__ __forceinline__ uint4 fresh16(const void *p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ int load_acquire(const int *p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// c[n] += rows (lo row, hi row of this lane) x tokens over this warp's share of
// `steps` 32-element steps.  SPLIT: the tokens' side is hi + lo.
template <typename T, int NT, bool SPLIT>
__device__ __forceinline__ void contract(float (&c)[NT][4], const T *r0, const T *r1, const T *const (&tok)[NT],
                                         const T *const (&tok2)[NT], int len, int warp, int q) {
  constexpr int U = NT == 1 ? 4 : 2;  // steps in flight
  constexpr bool BF = Two<T>::kBf;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * 32; k0 < len; k0 += 32 * kWarps * U) {
    uint4 A0[U], A1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 * kWarps + q * 8;
      A0[u] = r0 && k < len ? stream16(r0 + k) : zero;
      A1[u] = r1 && k < len ? stream16(r1 + k) : zero;
    }
    uint4 B[U][NT], B2[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 * kWarps + q * 8;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool in = tok[n] && k < len;
        if (SPLIT) {
          B[u][n] = in ? fresh16(tok[n] + k) : zero;
          B2[u][n] = in ? fresh16(tok2[n] + k) : zero;
        } else {
          B[u][n] = in ? __ldg(reinterpret_cast<const uint4 *>(tok[n] + k)) : zero;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816<BF>(c[n], A0[u].x, A1[u].x, A0[u].y, A1[u].y, B[u][n].x, B[u][n].y);
        mma16816<BF>(c[n], A0[u].z, A1[u].z, A0[u].w, A1[u].w, B[u][n].z, B[u][n].w);
        if (SPLIT) {
          mma16816<BF>(c[n], A0[u].x, A1[u].x, A0[u].y, A1[u].y, B2[u][n].x, B2[u][n].y);
          mma16816<BF>(c[n], A0[u].z, A1[u].z, A0[u].w, A1[u].w, B2[u][n].z, B2[u][n].w);
        }
      }
    }
  }
}

constexpr int kMaxNT = 4;  // tokens of one pass over a unit's weights: 32

struct ExpertSmem {
  float red[kWarps][kMaxNT][16][8];
  int first[kMaxExperts + 1];          // an expert's entries in `slots`
  int fill[kMaxExperts];
  int active[kMaxExperts];
  unsigned short slots[kMaxTokens * kMaxTopK];  // token * k + choice, by expert
  int n_active, ticket, last, ok;
};

template <typename T, int NT, bool DOWN>
__device__ __forceinline__ void unit_pass(const MoeArgs &a, ExpertSmem &sm, int e, int base, int count, int row0,
                                          int lane, int warp) {
  constexpr bool BF = Two<T>::kBf;
  const int g = lane >> 2, q = lane & 3;
  const T *r0, *r1;
  const int len = DOWN ? a.F : a.d;
  if (DOWN) {
    const T *w = static_cast<const T *>(a.w_out) + (size_t)e * a.d * a.F;
    r0 = row0 + g < a.d ? w + (size_t)(row0 + g) * a.F : nullptr;
    r1 = row0 + 8 + g < a.d ? w + (size_t)(row0 + 8 + g) * a.F : nullptr;
  } else {
    const T *w = static_cast<const T *>(a.w_in) + (size_t)e * 2 * a.F * a.d;
    r0 = w + (size_t)(row0 + g) * a.d;  // F is a multiple of 8: the rows exist
    r1 = w + (size_t)(a.F + row0 + g) * a.d;
  }
  const T *tok[NT], *tok2[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    tok[n] = tok2[n] = nullptr;
    if (n * 8 + g < count) {
      const int slot = sm.slots[base + n * 8 + g];
      if (DOWN) {
        tok[n] = static_cast<const T *>(a.hi) + (size_t)slot * a.F;
        tok2[n] = static_cast<const T *>(a.lo) + (size_t)slot * a.F;
      } else {
        tok[n] = static_cast<const T *>(a.x) + (size_t)(slot / a.k) * a.d;
      }
    }
  }
  float c[NT][4] = {};
  contract<T, NT, DOWN>(c, r0, r1, tok, tok2, len, warp, q);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2 *>(&sm.red[warp][n][g][2 * q]) = make_float2(c[n][0], c[n][1]);
    *reinterpret_cast<float2 *>(&sm.red[warp][n][g + 8][2 * q]) = make_float2(c[n][2], c[n][3]);
  }
  __syncthreads();
  if (DOWN) {
    for (int i = threadIdx.x; i < NT * 128; i += 32 * kWarps) {
      const int n = i >> 7, col = (i >> 4) & 7, row = i & 15;
      if (n * 8 + col < count && row0 + row < a.d) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sm.red[w][n][row][col];
        const int slot = sm.slots[base + n * 8 + col];
        a.part[(size_t)slot * a.d + row0 + row] = v * (a.weights[slot] * (BF ? 1.f : 1.f / kHalfScale));
      }
    }
  } else {
    for (int i = threadIdx.x; i < NT * 64; i += 32 * kWarps) {
      const int n = i >> 6, col = (i >> 3) & 7, row = i & 7;
      if (n * 8 + col < count) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          gate += sm.red[w][n][row][col];
          up += sm.red[w][n][row + 8][col];
        }
        const float act = a.act == FK_ACT_SILU ? gate / (1.f + expf(-gate))
                                               : 0.5f * gate * (1.f + erff(gate * 0.70710678118654752f));
        float h = act * up;
        if (!BF) h *= kHalfScale;
        const size_t at = (size_t)sm.slots[base + n * 8 + col] * a.F + row0 + row;
        const T hi = static_cast<T>(h);
        static_cast<T *>(a.hi)[at] = hi;
        static_cast<T *>(a.lo)[at] = static_cast<T>(h - static_cast<float>(hi));
      }
    }
  }
  __syncthreads();
}

template <typename T, bool DOWN>
__device__ __forceinline__ void unit(const MoeArgs &a, ExpertSmem &sm, int e, int row0, int lane, int warp) {
  const int end = sm.first[e + 1];
  for (int base = sm.first[e]; base < end; base += 8 * kMaxNT) {
    const int count = min(end - base, 8 * kMaxNT);
    if (count <= 8) unit_pass<T, 1, DOWN>(a, sm, e, base, count, row0, lane, warp);
    else if (count <= 16) unit_pass<T, 2, DOWN>(a, sm, e, base, count, row0, lane, warp);
    else unit_pass<T, 4, DOWN>(a, sm, e, base, count, row0, lane, warp);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps, 2) k_experts(const MoeArgs a) {
  extern __shared__ uint8_t expert_smem[];
  ExpertSmem &sm = *reinterpret_cast<ExpertSmem *>(expert_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slots = a.T * a.k;
  for (int e = tid; e < a.E; e += blockDim.x) sm.fill[e] = 0;
  __syncthreads();
  pdl_wait();
  for (int i = tid; i < slots; i += blockDim.x) atomicAdd(&sm.fill[a.ids[i]], 1);
  __syncthreads();
  if (warp == 0) {  // offsets, and the experts that any token chose
    int off = 0, act = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? sm.fill[e] : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (e < a.E) sm.first[e] = sm.fill[e] = off + inc - n;
      const unsigned some = __ballot_sync(0xffffffffu, n > 0);
      if (n > 0) sm.active[act + __popc(some & ((1u << lane) - 1u))] = e;
      act += __popc(some);
      off += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      sm.first[a.E] = off;
      sm.n_active = act;
    }
  }
  __syncthreads();
  for (int i = tid; i < slots; i += blockDim.x) sm.slots[atomicAdd(&sm.fill[a.ids[i]], 1)] = (unsigned short)i;
  if (tid == 0) sm.ticket = atomicAdd(a.tickets, 1);
  __syncthreads();

  const int ups = a.F / 8, downs = (a.d + 15) / 16;
  const int n_up = sm.n_active * ups, n_all = n_up + sm.n_active * downs;
  int *done_up = a.tickets + 1, *done_block = a.tickets + 1 + a.E;
  for (;;) {
    const int t = sm.ticket;
    __syncthreads();
    if (t >= n_all) return;
    int next = 0;
    if (tid == 0) next = atomicAdd(a.tickets, 1);  // in flight under this unit's loads
    if (t < n_up) {
      const int ae = t / ups, e = sm.active[ae];
      unit<T, false>(a, sm, e, (t - ae * ups) * 8, lane, warp);
      if (tid == 0) {
        __threadfence();
        atomicAdd(done_up + e, 1);
      }
    } else {
      const int ae = (t - n_up) / downs, blk = (t - n_up) - ae * downs, e = sm.active[ae];
      if (tid == 0) {
        int ok = 1;
        if (load_acquire(done_up + e) < ups) {
          const unsigned long long t0 = sm100::globaltimer();
          while (load_acquire(done_up + e) < ups) {
            if (sm100::globaltimer() - t0 > kWaitLimitNs) {
              atomicCAS(a.err, DEV_OK, DEV_TIMEOUT);
              ok = 0;
              break;
            }
          }
        }
        sm.ok = ok;
      }
      __syncthreads();
      if (!sm.ok) return;
      unit<T, true>(a, sm, e, blk * 16, lane, warp);
      if (tid == 0) {
        __threadfence();
        sm.last = atomicAdd(done_block + blk, 1) == sm.n_active - 1;
      }
      __syncthreads();
      if (sm.last) {
        __threadfence();
        // the block's 16 columns of y: the slots of each token, in order
        for (int i = tid; i < a.T * 16; i += blockDim.x) {
          const int tok = i >> 4, col = blk * 16 + (i & 15);
          if (col < a.d) {
            float v = 0.f;
            for (int j = 0; j < a.k; ++j) v += __ldcg(a.part + (size_t)(tok * a.k + j) * a.d + col);
            static_cast<T *>(a.y)[(size_t)tok * a.d + col] = static_cast<T>(v);
          }
        }
      }
    }
    if (tid == 0) sm.ticket = next;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side
int check_moe(const fk_moe_shape *m) {
  if (!m) return set_error(FK_EINVAL, "shape is NULL");
  if (m->dtype == FK_F32) return set_error(FK_EUNSUPPORTED, "fk_moe takes fp16 or bf16");
  if (m->dtype != FK_F16 && m->dtype != FK_BF16)
    return set_error(FK_EINVAL, "unknown dtype " + std::to_string(m->dtype));
  if (m->T < 0 || m->E <= 0 || m->d <= 0 || m->F <= 0) return set_error(FK_EINVAL, "T must be >= 0, E, d and F positive");
  if (m->d % 8 || m->F % 8) return set_error(FK_EINVAL, "d and F must be multiples of 8 (16-byte rows)");
  if (m->top_k < 1 || m->top_k > m->E) return set_error(FK_EINVAL, "top_k must be in [1, E]");
  if (m->act != FK_ACT_SILU && m->act != FK_ACT_GELU) return set_error(FK_EINVAL, "unknown activation");
  if (m->T > kMaxTokens || m->E > kMaxExperts || m->top_k > kMaxTopK)
    return set_error(FK_EUNSUPPORTED, "more than 256 tokens, 512 experts or 16 experts per token");
  if (m->d > (1 << 20) || m->F > (1 << 20)) return set_error(FK_EUNSUPPORTED, "d or F above 2^20");
  return FK_OK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

int moe_counters(const fk_moe_shape &m) { return 1 + m.E + (m.d + 15) / 16; }

size_t moe_bytes(const fk_moe_shape &m) {
  const size_t slots = (size_t)m.T * m.top_k;
  return round256((size_t)moe_counters(m) * 4) + 2 * round256(slots * m.F * 2) + round256(slots * m.d * 4);
}

template <typename T>
int launch_moe(const MoeArgs &a, cudaStream_t s) {
  FK_CUDA(launch_pdl(k_route<T>, dim3((a.T + kRouteCtas - 1) / kRouteCtas * kRouteCtas), dim3(32 * kWarps), 0, s, a));
  FK_TRY(launched());
  FK_TRY(set_smem_limit((const void *)k_experts<T>, (int)sizeof(ExpertSmem)));
  const long long units = (long long)std::min(a.E, a.T * a.k) * (a.F / 8 + (a.d + 15) / 16);
  const int grid = (int)std::min<long long>(2LL * num_sms(), units);
  FK_CUDA(launch_pdl(k_experts<T>, dim3(grid), dim3(32 * kWarps), sizeof(ExpertSmem), s, a));
  return launched();
}

}  // namespace
}  // namespace fk

using namespace fk;

extern "C" {

int fk_moe_workspace(const fk_moe_shape *shape, long long *bytes) {
  FK_TRY(check_moe(shape));
  if (!bytes) return set_error(FK_EINVAL, "bytes is NULL");
  *bytes = (long long)moe_bytes(*shape);
  return FK_OK;
}

int fk_moe(const fk_moe_shape *shape, const void *x, const void *router, const void *w_in, const void *w_out, void *y,
           int32_t *expert_ids, float *expert_weights, void *workspace, long long workspace_bytes,
           fk_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FK_TRY(check_moe(shape));
  const fk_moe_shape m = *shape;
  if (m.T == 0) return FK_OK;
  FK_TRY(check_ptr(x, "x", true));
  FK_TRY(check_ptr(router, "router", true));
  FK_TRY(check_ptr(w_in, "w_in", true));
  FK_TRY(check_ptr(w_out, "w_out", true));
  FK_TRY(check_ptr(y, "y", false));
  FK_TRY(check_ptr(expert_ids, "expert_ids", false));
  FK_TRY(check_ptr(expert_weights, "expert_weights", false));
  FK_TRY(check_ptr(workspace, "workspace", true));
  if (workspace_bytes < (long long)moe_bytes(m))
    return set_error(FK_EINVAL, "workspace is smaller than fk_moe_workspace asks for");
  FK_TRY(check_dev(x, "x"));
  FK_TRY(check_dev(router, "router"));
  FK_TRY(check_dev(w_in, "w_in"));
  FK_TRY(check_dev(w_out, "w_out"));
  FK_TRY(check_dev(y, "y"));
  FK_TRY(check_dev(expert_ids, "expert_ids"));
  FK_TRY(check_dev(expert_weights, "expert_weights"));
  FK_TRY(check_dev(workspace, "workspace"));
  MoeArgs a = {};
  a.T = m.T, a.E = m.E, a.d = m.d, a.F = m.F, a.k = m.top_k, a.act = m.act, a.renorm = m.renormalize != 0;
  a.x = x, a.router = router, a.w_in = w_in, a.w_out = w_out, a.y = y;
  a.ids = expert_ids, a.weights = expert_weights;
  const size_t slots = (size_t)m.T * m.top_k;
  a.counters = moe_counters(m);
  char *w = static_cast<char *>(workspace);
  a.tickets = reinterpret_cast<int *>(w);
  w += round256((size_t)a.counters * 4);
  a.hi = w;
  w += round256(slots * m.F * 2);
  a.lo = w;
  w += round256(slots * m.F * 2);
  a.part = reinterpret_cast<float *>(w);
  FK_TRY(soft_error_word(&a.err));
  if (m.dtype == FK_BF16) return launch_moe<__nv_bfloat16>(a, s);
  return launch_moe<__half>(a, s);
}

}  // extern "C"
