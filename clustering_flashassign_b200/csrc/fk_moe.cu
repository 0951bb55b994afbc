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
// k_route: one cluster of 8 CTAs per 4 tokens.  The CTAs share the experts; a
// thread keeps its slice of the 4 tokens in registers and meets every expert's
// row with it.  Scores are summed in fp64 (products of 16-bit values are exact,
// so experts are ranked by their exact scores) and sent to the CTA of their
// token, which ranks the experts by counting the better ones.
//
// k_experts: a persistent kernel over units of weights, taken from a ticket
// counter in the order  gate/up of expert 0, 1, ..., down of expert 0, 1, ...
//   gate/up unit   8 gate rows and the 8 up rows of the same columns: the 16
//                  rows of one mma.sync m16n8k16, whose 8 columns are tokens,
//   down unit      16 rows of Wd against the expert's h.
// A unit belongs to a group of 1, 2, 4 or 8 warps that split its contraction:
// as few as still give every warp of the GPU something to do.  One warp per
// unit needs no barrier and no joining and streams on its own; with few units
// (one token) the split keeps enough loads in flight.
// A lane loads 16 consecutive bytes of a row; the contraction's order inside a
// 32-element step is free, so these 8 elements feed two MMA steps without a
// transpose.  (tcgen05 has nothing to offer here: 128 rows of weights would
// meet 8 token columns, and the weights would take a detour through shared
// memory; the register path streams them at the rate HBM gives.)
// A down unit waits until its expert's h is complete.  Tickets make that safe
// without a grid-wide barrier or a cooperative launch: whoever waits holds a
// later ticket than every unit it waits for, and those are held by warps that
// run already and do not wait themselves.  Products of the k experts are
// written per (token, slot) and the group that finishes a block of 16 output
// columns sums its slots in order, so results do not depend on the order of
// arrival.
//
// h is held in two parts of the weights' type, so that rounding it does not add
// to the result's own rounding: hi + lo in bf16 (16 significant bits), and in
// fp16 h / 64 = hi + lo / 2^11 (22 bits).  The division keeps the type's range
// ahead of h (|h| up to 4.19e6; beyond, h counts as infinite), and what hi
// leaves is at most 2^-11 of it, so lo at 2^11 times its size fits and stays off
// the type's lower end: small h are off by 2^-30 at most (unscaled, 2^-19: 1% of
// the result where gate and up products are near 0.01).  lo's products are
// summed on their own and join with the factor 2^-11.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fk_sm100.cuh"

namespace fk {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxTokens = 256;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;
constexpr int kRouteCtas = 8;  // CTAs of a cluster
constexpr int kRouteTokens = 4;  // its tokens
constexpr int kWarps = 8;
constexpr float kHalfScale = 1.f / 64.f;  // fp16: of h
constexpr float kLowScale = 2048.f;       // fp16: of what hi leaves of h

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
  int S;  // warps per unit
  long long early;  // bytes of w_in asked for before the routing is known
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
constexpr int kPerCta = kMaxExperts / kRouteCtas;  // experts of one CTA at most
constexpr int kRouteBatch = 4;                     // router rows worked on together

// Order of a score as an integer; NaN ranks with -inf, below everything else.
__device__ __forceinline__ unsigned long long score_key(double v) {
  if (!(v == v)) return 0ull;
  const long long b = __double_as_longlong(v == 0.0 ? 0.0 : v);
  const unsigned long long k = b < 0 ? ~(unsigned long long)b : (unsigned long long)b | (1ull << 63);
  return v == -INFINITY ? 0ull : k;
}

// Two CTAs an SM (128 registers): above 72 tokens the clusters no longer find room
// at once otherwise (256 tokens of 512 experts, d 2048: the layer 305 us against 336).
template <typename T>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(32 * kWarps, 2) k_route(const MoeArgs a) {
  __shared__ double part[kWarps][kPerCta][kRouteTokens];
  __shared__ double scores[kMaxExperts];
  __shared__ unsigned long long keys[kMaxExperts];
  __shared__ int sel[kMaxTopK];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = (int)cluster.block_rank();
  const int t0 = (blockIdx.x / kRouteCtas) * kRouteTokens;
  const int nt = min(kRouteTokens, a.T - t0);
  pdl_wait();
  pdl_trigger();
  for (int i = blockIdx.x * blockDim.x + tid; i < a.counters; i += gridDim.x * blockDim.x) a.tickets[i] = 0;
  const T *xs = static_cast<const T *>(a.x) + (size_t)t0 * a.d;
  const T *rs = static_cast<const T *>(a.router);
  const int mine = a.E > cta ? (a.E - cta + kRouteCtas - 1) / kRouteCtas : 0;  // experts cta, cta + 8, ...
  for (int k0 = 0; k0 < a.d; k0 += 8 * 32 * kWarps) {
    const int k = k0 + tid * 8;
    double x[kRouteTokens][8];
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
      if (t < nt) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < a.d) v = *reinterpret_cast<const uint4 *>(xs + (size_t)t * a.d + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = Two<T>::f(w[j]);
          x[t][2 * j] = f.x;
          x[t][2 * j + 1] = f.y;
        }
      }
    }
    uint4 r[kRouteBatch];
    auto fetch = [&](int e0) {
#pragma unroll
      for (int i = 0; i < kRouteBatch; ++i) {
        r[i] = make_uint4(0, 0, 0, 0);
        if (e0 + i < mine && k < a.d)
          r[i] = *reinterpret_cast<const uint4 *>(rs + (size_t)(cta + (e0 + i) * kRouteCtas) * a.d + k);
      }
    };
    fetch(0);
    for (int e0 = 0; e0 < mine; e0 += kRouteBatch) {
      // the experts of a batch are independent chains of fp64 additions
      double acc[kRouteBatch][kRouteTokens] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < kRouteBatch; ++i) {
          const uint32_t w = j == 0 ? r[i].x : j == 1 ? r[i].y : j == 2 ? r[i].z : r[i].w;
          const float2 f = Two<T>::f(w);
          const double lo = f.x, hi = f.y;
#pragma unroll
          for (int t = 0; t < kRouteTokens; ++t)
            if (t < nt) acc[i][t] = fma(x[t][2 * j + 1], hi, fma(x[t][2 * j], lo, acc[i][t]));
        }
      }
      if (e0 + kRouteBatch < mine) fetch(e0 + kRouteBatch);
      if (nt == 1) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
          for (int i = 0; i < kRouteBatch; ++i) acc[i][0] += __shfl_xor_sync(0xffffffffu, acc[i][0], o);
      } else {
        // four sums over 32 lanes: two exchanges halve the tokens a lane carries,
        // three more add up the eight copies; lanes 0, 8, 16, 24 hold one each
#pragma unroll
        for (int o = 2; o; o >>= 1) {
          const bool up = lane & (o * 8);
#pragma unroll
          for (int t = 0; t < o; ++t)
#pragma unroll
            for (int i = 0; i < kRouteBatch; ++i) {
              const double keep = up ? acc[i][t + o] : acc[i][t], give = up ? acc[i][t] : acc[i][t + o];
              acc[i][t] = keep + __shfl_xor_sync(0xffffffffu, give, o * 8);
            }
        }
#pragma unroll
        for (int o = 4; o; o >>= 1)
#pragma unroll
          for (int i = 0; i < kRouteBatch; ++i) acc[i][0] += __shfl_xor_sync(0xffffffffu, acc[i][0], o);
      }
      // nt == 1: lane 0 holds the sum (of token 0); else lanes 0, 8, 16, 24
      if ((lane & 7) == 0 && (nt > 1 || lane == 0)) {
#pragma unroll
        for (int i = 0; i < kRouteBatch; ++i)
          if (e0 + i < mine) {
            double *out = &part[warp][e0 + i][lane >> 3];
            *out = k0 ? *out + acc[i][0] : acc[i][0];
          }
      }
    }
  }
  __syncthreads();
  cluster.sync();  // every CTA of the cluster runs before its memory is written
  for (int i = tid; i < mine * kRouteTokens; i += blockDim.x) {
    const int e = i / kRouteTokens, t = i % kRouteTokens;
    if (t < nt) {
      double v = 0.0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[w][e][t];
      *cluster.map_shared_rank(scores + cta + e * kRouteCtas, t) = v;
    }
  }
  cluster.sync();
  if (cta >= nt) return;
  for (int e = tid; e < a.E; e += blockDim.x) keys[e] = score_key(scores[e]);
  __syncthreads();
  for (int e = tid; e < a.E; e += blockDim.x) {
    const unsigned long long key = keys[e];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < a.E; ++i) rank += keys[i] > key || (keys[i] == key && i < e);
    if (rank < a.k) sel[rank] = e;
  }
  __syncthreads();
  if (warp != 0) return;
  const double big = scores[sel[0]];
  const float p = lane < a.k ? expf((float)(scores[sel[lane]] - big)) : 0.f;
  float all = p;
  bool nan = false;
  if (!a.renorm) all = 0.f;
  for (int e = lane; e < a.E; e += 32) {
    nan |= !(scores[e] == scores[e]);
    if (!a.renorm) all += expf((float)(scores[e] - big));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  nan = __any_sync(0xffffffffu, nan);
  if (lane < a.k) {
    a.ids[(t0 + cta) * a.k + lane] = sel[lane];
    a.weights[(t0 + cta) * a.k + lane] = nan ? NAN : p / all;
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

// c[n] += rows (lo row, hi row of this lane) x tokens over the 32-element
// steps sub, sub + S, ... of a group of S warps.  SPLIT: the tokens' side is in two parts.
template <typename T, int NT, bool SPLIT>
__device__ __forceinline__ void contract(float (&c)[NT][4], const T *r0, const T *r1, const T *const (&tok)[NT],
                                         const T *const (&tok2)[NT], int len, int sub, int S, int q) {
  constexpr int U = NT == 1 ? (SPLIT ? 4 : 6) : NT == 2 ? 3 : 2;  // steps in flight
  constexpr bool BF = Two<T>::kBf;
  constexpr bool APART = SPLIT && !BF;  // the second part has a scale of its own
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int step = 32 * S;
  float low[APART ? NT : 1][4] = {};
  for (int k0 = sub * 32 + q * 8; k0 < len + q * 8; k0 += step * U) {
    uint4 A0[U], A1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      A0[u] = r0 && k < len ? stream16(r0 + k) : zero;
      A1[u] = r1 && k < len ? stream16(r1 + k) : zero;
    }
    uint4 B[U][NT], B2[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
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
          float(&c2)[4] = APART ? low[APART ? n : 0] : c[n];
          mma16816<BF>(c2, A0[u].x, A1[u].x, A0[u].y, A1[u].y, B2[u][n].x, B2[u][n].y);
          mma16816<BF>(c2, A0[u].z, A1[u].z, A0[u].w, A1[u].w, B2[u][n].z, B2[u][n].w);
        }
      }
    }
  }
  if constexpr (APART) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[n][i] = fmaf(low[n][i], 1.f / kLowScale, c[n][i]);
  }
}

constexpr int kMaxNT = 4;  // tokens of one pass over a unit's weights: 32

struct ExpertSmem {
  float red[kWarps][kMaxNT][4][32];    // a warp's accumulators, where warps share a unit
  int fill[kMaxExperts];
  int active[kMaxExperts];             // the experts that any token chose
  int first[kMaxExperts + 1];          // their entries in `slots`
  unsigned short slots[kMaxTokens * kMaxTopK];  // token * k + choice, by expert
  int n_active;
  int word[kWarps];                    // a group's ticket or verdict, handed to its warps
};

// A group of S consecutive warps of the CTA.
struct Group {
  int S, id, sub, lane;
  __device__ __forceinline__ bool leader() const { return sub == 0 && lane == 0; }
  __device__ __forceinline__ void sync() const {
    if (S == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(S * 32) : "memory");
  }
  // every thread of the group gets the leader's value
  __device__ __forceinline__ int share(ExpertSmem &sm, int v) const {
    if (S == 1) {
      v = __shfl_sync(0xffffffffu, v, 0);
      __syncwarp();  // the exchange orders no memory: what the leader has seen, the others see from here on
      return v;
    }
    if (leader()) sm.word[id] = v;
    sync();
    const int r = *(volatile int *)&sm.word[id];
    sync();
    return r;
  }
};

__device__ __forceinline__ float activate(int act, float g) {
  return act == FK_ACT_SILU ? g / (1.f + expf(-g)) : 0.5f * g * (1.f + erff(g * 0.70710678118654752f));
}

template <typename T, int NT, bool DOWN>
__device__ __forceinline__ void unit_pass(const MoeArgs &a, ExpertSmem &sm, const Group &gr, int e, int base, int count,
                                          int row0) {
  constexpr bool BF = Two<T>::kBf;
  const int g = gr.lane >> 2, q = gr.lane & 3;
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
  contract<T, NT, DOWN>(c, r0, r1, tok, tok2, len, gr.sub, gr.S, q);
  if (gr.S > 1) {  // the group's first warps take one tile of 8 tokens each and add up its parts
    const int w0 = gr.id * gr.S;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sm.red[w0 + gr.sub][n][i][gr.lane] = c[n][i];
    gr.sync();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n % gr.S != gr.sub) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = 0.f;
        for (int w = 0; w < gr.S; ++w) v += sm.red[w0 + w][n][i][gr.lane];
        c[n][i] = v;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (gr.S > 1 && n % gr.S != gr.sub) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // this lane: rows g (c[n][i]) and g + 8 (c[n][2 + i]) of token 2 q + i
      const int col = n * 8 + 2 * q + i;
      if (col < count) {
        const int slot = sm.slots[base + col];
        if (DOWN) {
          const float w = a.weights[slot] * (BF ? 1.f : 1.f / kHalfScale);
          float *out = a.part + (size_t)slot * a.d + row0 + g;
          if (row0 + g < a.d) out[0] = c[n][i] * w;
          if (row0 + 8 + g < a.d) out[8] = c[n][2 + i] * w;
        } else {
          float h = activate(a.act, c[n][i]) * c[n][2 + i];
          if (!BF) h *= kHalfScale;
          const size_t at = (size_t)slot * a.F + row0 + g;
          const T hi = static_cast<T>(h);
          const float left = fabsf(static_cast<float>(hi)) < INFINITY ? h - static_cast<float>(hi) : 0.f;
          static_cast<T *>(a.hi)[at] = hi;
          static_cast<T *>(a.lo)[at] = static_cast<T>(BF ? left : left * kLowScale);
        }
      }
    }
  }
  gr.sync();
}

template <typename T, bool DOWN>
__device__ __forceinline__ void unit(const MoeArgs &a, ExpertSmem &sm, const Group &gr, int ae, int row0) {
  const int e = sm.active[ae], end = sm.first[ae + 1];
  for (int base = sm.first[ae]; base < end; base += 8 * kMaxNT) {
    const int count = min(end - base, 8 * kMaxNT);
    if (count <= 8) unit_pass<T, 1, DOWN>(a, sm, gr, e, base, count, row0);
    else if (count <= 16) unit_pass<T, 2, DOWN>(a, sm, gr, e, base, count, row0);
    else unit_pass<T, 4, DOWN>(a, sm, gr, e, base, count, row0);
  }
}

// The chosen experts, by index, and their (token, choice) entries.  Every CTA
// has the same list of experts, since tickets number them.
__device__ __forceinline__ void list_experts(const MoeArgs &a, ExpertSmem &sm, int tid, int lane, int warp) {
  const int slots = a.T * a.k;
  if (slots <= 32) {  // one warp, a lane per entry
    if (warp == 0) {
      const int e = lane < slots ? a.ids[lane] : -1;
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      const bool lead = lane < slots && (__ffs(peers) - 1) == lane;
      const unsigned leads = __ballot_sync(0xffffffffu, lead);
      // the chosen experts of lower index, and their entries
      int off = 0, ae = 0;
      for (unsigned m = leads; m; m &= m - 1) {
        const int l = __ffs(m) - 1, other = __shfl_sync(0xffffffffu, e, l);
        const unsigned p = __shfl_sync(0xffffffffu, peers, l);
        if (other < e) {
          off += __popc(p);
          ++ae;
        }
      }
      if (lead) {
        sm.active[ae] = e;
        sm.first[ae] = off;
      }
      if (lane < slots) sm.slots[off + __popc(peers & ((1u << lane) - 1u))] = (unsigned short)lane;
      if (lane == 0) {
        sm.n_active = __popc(leads);
        sm.first[__popc(leads)] = slots;
      }
    }
    __syncthreads();
    return;
  }
  for (int i = tid; i < slots; i += blockDim.x) atomicAdd(&sm.fill[a.ids[i]], 1);
  __syncthreads();
  if (warp == 0) {
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
      if (e < a.E) sm.fill[e] = off + inc - n;
      const unsigned some = __ballot_sync(0xffffffffu, n > 0);
      if (n > 0) {
        const int ae = act + __popc(some & ((1u << lane) - 1u));
        sm.active[ae] = e;
        sm.first[ae] = off + inc - n;
      }
      act += __popc(some);
      off += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      sm.first[act] = off;
      sm.n_active = act;
    }
  }
  __syncthreads();
  for (int i = tid; i < slots; i += blockDim.x) sm.slots[atomicAdd(&sm.fill[a.ids[i]], 1)] = (unsigned short)i;
  __syncthreads();
}

// Columns [blk * 16, + 16) of y: the slots of each token, in order.  A lane
// takes four columns (d is a multiple of 8).
template <typename T>
__device__ __forceinline__ void sum_slots(const MoeArgs &a, const Group &gr, int blk) {
  const int who = gr.sub * 32 + gr.lane, col = blk * 16 + (who & 3) * 4;
  if (col >= a.d) return;
  for (int t = who >> 2; t < a.T; t += 8 * gr.S) {
    const float *p = a.part + (size_t)t * a.k * a.d + col;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < a.k; ++j) {
      const float4 w = __ldcg(reinterpret_cast<const float4 *>(p + (size_t)j * a.d));
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    T *y = static_cast<T *>(a.y) + (size_t)t * a.d + col;
    y[0] = static_cast<T>(v.x);
    y[1] = static_cast<T>(v.y);
    y[2] = static_cast<T>(v.z);
    y[3] = static_cast<T>(v.w);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps, 2) k_experts(const MoeArgs a) {
  extern __shared__ uint8_t expert_smem[];
  ExpertSmem &sm = *reinterpret_cast<ExpertSmem *>(expert_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Group gr = {a.S, warp / a.S, warp % a.S, lane};
  for (int e = tid; e < a.E; e += blockDim.x) sm.fill[e] = 0;
  __syncthreads();
  // where most experts will be chosen, the first units' weights are known
  // before the routing is: they travel to L2 meanwhile
  for (long long o = ((long long)blockIdx.x * blockDim.x + tid) * 128; o < a.early; o += (long long)gridDim.x * blockDim.x * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(a.w_in) + o));
  pdl_wait();
  int t = 0;
  if (gr.leader()) t = atomicAdd(a.tickets, 1);  // in flight while the lists are made
  list_experts(a, sm, tid, lane, warp);

  const int ups = a.F / 8, downs = (a.d + 15) / 16;
  const int n_up = sm.n_active * ups, n_all = n_up + sm.n_active * downs;
  int *done_up = a.tickets + 1, *done_block = a.tickets + 1 + a.E;
  t = gr.share(sm, t);
  while (t < n_all) {
    int next = 0;
    if (gr.leader()) next = atomicAdd(a.tickets, 1);  // in flight under this unit's loads
    if (t < n_up) {
      const int ae = t / ups;
      unit<T, false>(a, sm, gr, ae, (t - ae * ups) * 8);
      if (gr.leader()) {
        __threadfence();
        atomicAdd(done_up + ae, 1);
      }
    } else {
      const int ae = (t - n_up) / downs, blk = (t - n_up) - ae * downs;
      int ok = 1;
      if (gr.leader() && load_acquire(done_up + ae) < ups) {
        const unsigned long long t0 = sm100::globaltimer();
        while (load_acquire(done_up + ae) < ups) {
          if (sm100::globaltimer() - t0 > kWaitLimitNs) {
            atomicCAS(a.err, DEV_OK, DEV_TIMEOUT);
            ok = 0;
            break;
          }
        }
      }
      if (!gr.share(sm, ok)) return;
      unit<T, true>(a, sm, gr, ae, blk * 16);
      int last = 0;
      if (gr.leader()) {
        __threadfence();
        last = atomicAdd(done_block + blk, 1) == sm.n_active - 1;
        __threadfence();
      }
      if (gr.share(sm, last)) sum_slots<T>(a, gr, blk);
    }
    t = gr.share(sm, next);
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
  FK_CUDA(launch_pdl(k_route<T>, dim3((a.T + kRouteTokens - 1) / kRouteTokens * kRouteCtas), dim3(32 * kWarps), 0, s, a));
  FK_TRY(launched());
  FK_TRY(set_smem_limit((const void *)k_experts<T>, (int)sizeof(ExpertSmem)));
  // the fewest warps per unit that give every warp of the grid one, for as many
  // experts as even choices would hit
  const double hit = a.E * (1.0 - std::pow(1.0 - (double)a.k / a.E, a.T));
  const long long fewer = (long long)(hit * std::min(a.F / 8, (a.d + 15) / 16));
  const long long units = (long long)std::min(a.E, a.T * a.k) * (a.F / 8 + (a.d + 15) / 16);
  const int grid = (int)std::min<long long>(2LL * num_sms(), units);
  MoeArgs b = a;
  b.S = 1;
  const long long w_in = 4LL * a.E * a.F * a.d;
  b.early = hit >= 0.85 * a.E ? std::min(w_in, 32LL << 20) : 0;
  while (b.S < kWarps && fewer * b.S < (long long)grid * kWarps) b.S *= 2;
  FK_CUDA(launch_pdl(k_experts<T>, dim3(grid), dim3(32 * kWarps), sizeof(ExpertSmem), s, b));
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
