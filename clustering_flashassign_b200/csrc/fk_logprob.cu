// Token log probabilities (the soft form of the assignment) and their
// gradients.
//
//   s_nk  = scale * x_n . c_k + bias_k
//   lse_n = log sum_k exp(s_nk),  p_nk = exp(s_nk - lse_n)
//   logp_n = s_{n, id_n} - lse_n,  H_n = -sum_k p_nk log p_nk
//   top:  the largest s_nk, lowest k on ties
//   G_nk  = dL/ds_nk = a_n (1[k = id_n] - p_nk) + l_n p_nk - e_n p_nk (log p_nk + H_n)
//           for the upstream gradients a, l, e of logp, lse and H,
//   dx = scale * G C,  dc = scale * G^T X,  dbias_k = sum_n G_nk.
//
// The (B, N, K) scores never reach memory in the forward pass, as the distance
// matrix never does in FlashAssign: every 128 x 256 tile of them is read once
// from TMEM by the epilogue, which keeps the running maximum, sum and
// sum e^{s-m}(s-m) (the entropy's) of each row and the row's best columns.
// Rows are split over column runs and joined by a second, small kernel.
// All row statistics are fp32, in base 2 (scale and bias carry log2 e).
//
// The backward pass recomputes each tile of scores, turns it into G rounded
// once to the operands' type (bf16: relative 2^-9 of each value; fp16: 2^-11
// after a power-of-two scale that brings the largest possible |G| of the call
// to 2^14; fp32: three bf16 planes, 2^-25), and multiplies G with C and X.
// G is held for a block of rows at a time, sized by a fixed budget.
// The column sums of dbias use G before the rounding.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fk_tile_engine.cuh"

namespace fk {
namespace {

using tile::Plan;
using tile::Unit;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;
// Below 2^-256 of the maximum a term is zero in fp32; the clamp keeps
// 0 * -inf out of the entropy sum and leaves NaN sums NaN.
constexpr float kLowest = -256.f;
// Columns beyond `top` that the running lists keep: the lists rank by fp32
// scores, and the final order is settled in fp64 among top + kSpare columns.
constexpr int kSpare = 4;
constexpr int kMaxTop = 28;  // top + kSpare candidates: one per lane of the joining warp
// One CTA's 128 rows hold all rows: the second half of a pair's 256-row tile
// would be empty, and single CTAs spread a short run of columns over all SMs.
// Otherwise pairs.
inline int group_of(long long rows) { return rows <= tile::kRows ? 1 : 2; }

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <typename T>
__device__ __forceinline__ float to_f(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v) { return static_cast<T>(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// A warp's bias of its half tile's 128 columns, times log2 e, in shared memory;
// columns past the last count as masked.  `masked`: which of the four
// 32-column chunks hold a masked column.
struct BiasTile {
  static constexpr int kFloats = 128;
  float *sb;
  unsigned masked = 0;
  __device__ __forceinline__ void load(const float *bias, long long col0, long long K, int lane) {
    __syncwarp();  // the previous tile's values have been read
    masked = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long col = col0 + i * 32 + lane;
      const float b = col < K ? __ldg(bias + col) : kNegInf;
      sb[i * 32 + lane] = b * kLog2e;
      if (__any_sync(0xffffffffu, b == kNegInf)) masked |= 1u << i;
    }
    __syncwarp();
  }
};

// The 32 scores (base 2) of a thread's row in columns [col, col + 32), chunk i
// of the half tile.  A bias of -inf masks its column whatever the product holds.
template <bool BIAS>
__device__ __forceinline__ void scores32(const float (&r)[32], float scale2, const BiasTile &bt, int i, long long col,
                                         long long K, float (&t)[32]) {
  if (BIAS) {
    const float4 *sb = reinterpret_cast<const float4 *>(bt.sb + i * 32);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 b = sb[j];
      t[4 * j] = fmaf(r[4 * j], scale2, b.x);
      t[4 * j + 1] = fmaf(r[4 * j + 1], scale2, b.y);
      t[4 * j + 2] = fmaf(r[4 * j + 2], scale2, b.z);
      t[4 * j + 3] = fmaf(r[4 * j + 3], scale2, b.w);
    }
    if (bt.masked >> i & 1u) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (bt.sb[i * 32 + j] == kNegInf) t[j] = kNegInf;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j] = r[j] * scale2;
    if (col + 32 > K) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j >= K) t[j] = kNegInf;
    }
  }
}

// ------------------------------------------------------------------ forward
struct StatArgs {
  float scale2;
  const float *bias;  // (B, K) or NULL
  const int32_t *ids;
  long long N, K;
  int parts;  // partial results per row: 2 * runs
  int L;      // columns kept per partial list, 0: none
  float4 *part;          // (B, N, parts): m, sum, sum e (t - m), target score
  float *top_v;          // (B, N, parts, L)
  int32_t *top_i;
};

// Running statistics of one row per thread.
//
// The sums refer to a maximum that follows the row's with a slack of 2^8: a
// chunk's exponentials then rarely wait for its maximum.
//
// The best columns.  Eight columns of which no row of the warp wants anything
// (their maximum beats none of the lists) cost a comparison.  Otherwise they
// are drained from their maximum downwards, every lane inserting its own best
// column in the same step, until no lane's remainder beats its list.  A list of
// 8 or 16 (LREG) sits in registers, where an insertion is a branchless shift of
// five instructions a place; a longer one in shared memory.
template <bool BIAS, bool TOP, int LREG, bool SEG>
struct StatEpi {
  using Args = StatArgs;
  static constexpr bool kSeg = SEG;
  static constexpr int kSlots = 32 * tile::kEpiWarps;
  static constexpr int kCap = LREG ? LREG : 1;
  const Args &a;
  const int r, half, slot, lane;
  BiasTile bt;
  float *lv;
  int32_t *li;
  const float *bias = nullptr;
  long long row = 0, at = 0;
  int id = -1;
  bool idle = false;  // none of the warp's rows exists
  float m = 0.f, sum = 0.f, us = 0.f, tgt = 0.f, thr = 0.f;
  float rv[kCap];
  int rk[kCap];

  __device__ StatEpi(const Args &args, int lane_, int r_in_tile, int half_, uint8_t *smem)
      : a(args), r(r_in_tile), half(half_), slot(half_ * 128 + r_in_tile), lane(lane_) {
    float *f = reinterpret_cast<float *>(smem);
    if (BIAS) {
      bt.sb = f + (slot / 32) * BiasTile::kFloats;
      f += tile::kEpiWarps * BiasTile::kFloats;
    }
    lv = f + slot;
    li = reinterpret_cast<int32_t *>(f) + args.L * kSlots + slot;
  }
  static size_t smem_bytes(int L) {
    return (BIAS ? tile::kEpiWarps * BiasTile::kFloats * 4 : 0) + (TOP && !LREG ? (size_t)L * kSlots * 8 : 0);
  }

  __device__ void begin(const Unit &w, long long row0) {
    row = row0 + r;
    idle = row0 + (r & ~31) >= a.N;
    at = w.b * a.N + row;
    id = row < a.N ? __ldg(a.ids + at) : -1;
    if (BIAS) bias = a.bias + w.b * a.K;
    m = thr = tgt = kNegInf;
    sum = us = 0.f;
    if (TOP) {
      if (LREG) {
#pragma unroll
        for (int j = 0; j < kCap; ++j) {
          rv[j] = kNegInf;
          rk[j] = -1;
        }
      } else {
        for (int j = 0; j < a.L; ++j) {
          lv[j * kSlots] = kNegInf;
          li[j * kSlots] = -1;
        }
      }
      if (row >= a.N) thr = INFINITY;  // a row beyond the last keeps nothing
    }
  }
  __device__ __forceinline__ void prepare(long long col0) {
    if (BIAS && !skip(col0)) bt.load(bias, col0, a.K, lane);
  }

  __device__ __forceinline__ void insert(float v, int k) {
    int p = a.L - 1;
    for (; p > 0; --p) {
      const float q = lv[(p - 1) * kSlots];
      if (!(q < v)) break;
      lv[p * kSlots] = q;
      li[p * kSlots] = li[(p - 1) * kSlots];
    }
    lv[p * kSlots] = v;
    li[p * kSlots] = k;
    thr = lv[(a.L - 1) * kSlots];
  }

  // Into the register list (descending; an equal value that came earlier, from
  // lower columns, stays ahead).  v = -inf inserts nothing.
  __device__ __forceinline__ void insert_reg(float v, int k) {
#pragma unroll
    for (int i = kCap - 1; i >= 0; --i) {
      const bool below = v > rv[i];
      const bool shift = i > 0 && v > rv[i > 0 ? i - 1 : 0];
      rk[i] = below ? (shift ? rk[i > 0 ? i - 1 : 0] : k) : rk[i];
      rv[i] = i > 0 ? fmaxf(rv[i], fminf(rv[i > 0 ? i - 1 : 0], v)) : fmaxf(rv[i], v);
    }
    if (row < a.N) thr = rv[kCap - 1];
  }

  // Eight consecutive columns, m8 their maximum.
  __device__ __forceinline__ void drain8(float *t, float m8, int col) {
    while (__any_sync(0xffffffffu, m8 > thr)) {
      const bool take = m8 > thr;
      int j8 = 8;
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (t[j] == m8) j8 = j;
      if (LREG) insert_reg(take ? m8 : kNegInf, col + j8);
      else if (take) insert(m8, col + j8);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == j8) t[j] = kNegInf;
      __syncwarp();
      m8 = max3(max3(t[0], t[1], t[2]), max3(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
    }
  }

  __device__ __forceinline__ void chunk(const float (&acc)[32], long long col, int i) {
    float t[32];
    scores32<BIAS>(acc, a.scale2, bt, i, col, a.K, t);
    float g[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float *v = t + 8 * q;
      g[q] = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
    }
    const float cm = max3(fmaxf(g[0], g[1]), g[2], g[3]);
    if (cm > m + 8.f) {  // always the case for the first finite chunk
      if (m != kNegInf) {
        const float f = ex2(m - cm);
        us = f * fmaf(m - cm, sum, us);
        sum *= f;
      }
      m = cm;
    }
    const float ms = m == kNegInf ? 0.f : m;
    float s0 = 0.f, s1 = 0.f, u0 = 0.f, u1 = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float d0 = t[j] - ms, d1 = t[j + 1] - ms;
      const float e0 = ex2(d0), e1 = ex2(d1);
      s0 += e0;
      s1 += e1;
      u0 = fmaf(e0, fmaxf(d0, kLowest), u0);
      u1 = fmaf(e1, fmaxf(d1, kLowest), u1);
    }
    sum += s0 + s1;
    us += u0 + u1;
    const unsigned rel = (unsigned)(id - (int)col);
    if (__any_sync(0xffffffffu, rel < 32u)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (rel == (unsigned)j) tgt = t[j];
    }
    if (TOP && __any_sync(0xffffffffu, cm > thr)) {
#pragma unroll
      for (int q = 0; q < 4; ++q) drain8(t + 8 * q, g[q], (int)col + 8 * q);
    }
  }

  __device__ void end(const Unit &w) {
    if (row >= a.N) return;
    const long long p = at * a.parts + w.run * 2 + half;
    a.part[p] = make_float4(m, sum, us, tgt);
    if (TOP && LREG) {
#pragma unroll
      for (int j = 0; j < kCap; j += 4) {
        reinterpret_cast<float4 *>(a.top_v + p * kCap)[j / 4] = make_float4(rv[j], rv[j + 1], rv[j + 2], rv[j + 3]);
        reinterpret_cast<int4 *>(a.top_i + p * kCap)[j / 4] = make_int4(rk[j], rk[j + 1], rk[j + 2], rk[j + 3]);
      }
    } else if (TOP) {
      for (int j = 0; j < a.L; ++j) {
        a.top_v[p * a.L + j] = lv[j * kSlots];
        a.top_i[p * a.L + j] = li[j * kSlots];
      }
    }
  }
  __device__ __forceinline__ bool skip(long long col) const { return idle || col >= a.K; }
};

// Joins a row's partial results (one warp per row).
struct JoinArgs {
  const float4 *part;
  const float *top_v;
  const int32_t *top_i;
  const int32_t *ids;
  const void *x, *c;
  const float *bias;
  float scale;
  long long rows, N, K;
  int d, parts, L, cands, top;  // L: length of a partial list; cands = min(K, L)
  bool vec;  // rows of x and c can be read 16 bytes at a time
  float *logp, *lse, *entropy, *top_logp;
  int32_t *top_ids;
  int *err;
};

__device__ __forceinline__ void join_stats(float &m, float &s, float &u, float m2, float s2, float u2) {
  const float mm = fmaxf(m, m2);
  const float ms = mm == kNegInf ? 0.f : mm;
  // an empty side has s = u = 0 and its (clamped) distance contributes nothing;
  // a NaN sum stays NaN
  const float d1 = fmaxf(m - ms, kLowest), d2 = fmaxf(m2 - ms, kLowest);
  const float f1 = ex2(m - ms), f2 = ex2(m2 - ms);
  u = f1 * fmaf(d1, s, u) + f2 * fmaf(d2, s2, u2);
  s = f1 * s + f2 * s2;
  m = mm;
}

// Scores of four columns in fp64, by LPR lanes, from the operands as given:
// products of 16-bit values are exact, and fp64 sums keep neighbours in rank
// apart that the fp32 accumulation cannot.
template <typename T, int LPR>
__device__ __forceinline__ void exact_scores(const T *x, const T *c, const float *bias, float scale, const int (&k)[4],
                                             int d, bool vec, int lane, double (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = 0.0;
  constexpr int V = 16 / sizeof(T);
  if (vec) {
#pragma unroll 2
    for (int j = lane; j < d / V; j += LPR) {
      T xv[V], cv[4][V];
      *reinterpret_cast<uint4 *>(xv) = __ldg(reinterpret_cast<const uint4 *>(x) + j);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(cv[i]) = __ldg(reinterpret_cast<const uint4 *>(c + (size_t)k[i] * d) + j);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const double xd = (double)to_f(xv[q]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = fma(xd, (double)to_f(cv[i][q]), s[i]);
      }
    }
  } else {
    for (int j = lane; j < d; j += LPR) {
      const double xd = (double)to_f(x[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = fma(xd, (double)to_f(c[(size_t)k[i] * d + j]), s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    s[i] *= (double)scale;
    if (bias) s[i] = bias[k[i]] == kNegInf ? (double)kNegInf : s[i] + (double)bias[k[i]];
  }
}

constexpr int kJoinWarps = 8;
constexpr int kNoCol = 0x7fffffff;

// One warp's joined lists (and the row's candidates with their exact scores)
// where eight warps share a row.
struct JoinRow {
  float m[kJoinWarps], s[kJoinWarps], u[kJoinWarps], tgt[kJoinWarps];
  float v[kJoinWarps][32];
  int k[kJoinWarps][32];
  int cand[32];
  double exact[32];
};

// The best L of the lanes' sorted lists (read through get(j, v, k)); lane j of
// the group keeps the j-th.
template <int LPR, class Get>
__device__ __forceinline__ void draw(int L, int lane, Get get, float &mv, int &mk) {
  int head = 0;
  float hv;
  int hk;
  get(0, hv, hk);
  mv = kNegInf;
  mk = -1;
  for (int j = 0; j < L; ++j) {
    float v = hk >= 0 ? hv : kNegInf;
    int k = hk >= 0 ? hk : kNoCol;
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) {
      const float v2 = __shfl_xor_sync(0xffffffffu, v, o);
      const int k2 = __shfl_xor_sync(0xffffffffu, k, o);
      if (v2 > v || (v2 == v && k2 < k)) {
        v = v2;
        k = k2;
      }
    }
    if (lane == j && k != kNoCol) {
      mv = v;
      mk = k;
    }
    if (hk == k) {
      ++head;
      hk = -1;
      if (head < L) get(head, hv, hk);
    }
  }
}

// LPR lanes of WPR warps per row.  (8, 1): many rows of few parts, four rows a
// warp; (32, 1); (32, 8): few rows, whose exact scores would otherwise be one
// warp's long chain of loads.
template <typename T, int LPR, int WPR>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join(const JoinArgs a) {
  extern __shared__ float join_smem[];
  __shared__ JoinRow sh;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & (LPR - 1);
  const int sub = WPR > 1 ? warp : 0;  // this warp among the row's warps
  const long long per_block = WPR > 1 ? 1 : kJoinWarps * (32 / LPR);
  const long long r0 = (long long)blockIdx.x * per_block + (WPR > 1 ? 0 : threadIdx.x / LPR);
  // lanes of a row beyond the last one follow along on the last row
  const bool live = r0 < a.rows;
  const long long r = live ? r0 : a.rows - 1;
  const long long b = r / a.N;
  const int first = sub * LPR + lane, step = LPR * WPR;
  float m = kNegInf, s = 0.f, u = 0.f, tgt = kNegInf;
  for (int p = first; p < a.parts; p += step) {
    const float4 q = a.part[r * a.parts + p];
    join_stats(m, s, u, q.x, q.y, q.z);
    tgt = fmaxf(tgt, q.w);
  }
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float u2 = __shfl_xor_sync(0xffffffffu, u, o);
    // both sides join in the same order, so that all lanes hold the same bits
    if (lane & o) {
      float mm = m2, ss = s2, uu = u2;
      join_stats(mm, ss, uu, m, s, u);
      m = mm, s = ss, u = uu;
    } else {
      join_stats(m, s, u, m2, s2, u2);
    }
    tgt = fmaxf(tgt, __shfl_xor_sync(0xffffffffu, tgt, o));
  }
  if (WPR > 1) {
    if (lane == 0) {
      sh.m[warp] = m, sh.s[warp] = s, sh.u[warp] = u, sh.tgt[warp] = tgt;
    }
    __syncthreads();
    m = sh.m[0], s = sh.s[0], u = sh.u[0], tgt = sh.tgt[0];
    for (int w = 1; w < WPR; ++w) {
      join_stats(m, s, u, sh.m[w], sh.s[w], sh.u[w]);
      tgt = fmaxf(tgt, sh.tgt[w]);
    }
  }
  // a row whose columns are all masked has lse = -inf and an entropy of zero
  const bool none = m == kNegInf && s == 0.f;
  const float ls = log2f(s);
  if (live && lane == 0 && sub == 0) {
    const int id = a.ids[r];
    const bool valid = id >= 0 && id < a.K;
    if (id >= a.K) atomicCAS(a.err, DEV_OK, DEV_BAD_ID);
    a.lse[r] = none ? kNegInf : (m + ls) * kLn2;
    if (a.entropy) a.entropy[r] = none ? 0.f : (ls - u / s) * kLn2;
    a.logp[r] = !valid ? 0.f : (none || (tgt == kNegInf && s == s)) ? kNegInf : ((tgt - m) - ls) * kLn2;
  }
  if (a.top == 0) return;

  float mv;
  int mine;
  if (a.parts <= step) {  // one list per lane at most: drawn from where it lies
    const long long o = (r * a.parts + first) * a.L;
    draw<LPR>(a.L, lane,
              [&](int j, float &v, int &k) {
                k = -1;
                if (first < a.parts) {
                  v = __ldg(a.top_v + o + j);
                  k = __ldg(a.top_i + o + j);
                }
              },
              mv, mine);
  } else {  // each lane joins the lists of its parts into one of its own first
    float *lv = join_smem + (size_t)(threadIdx.x / LPR) * 2 * LPR * a.L + lane;
    int32_t *li = reinterpret_cast<int32_t *>(join_smem + (size_t)(threadIdx.x / LPR) * 2 * LPR * a.L + LPR * a.L) + lane;
    for (int j = 0; j < a.L; ++j) li[LPR * j] = -1;
    for (int p = first; p < a.parts; p += step) {
      const long long o = (r * a.parts + p) * a.L;
      for (int j = 0; j < a.L; ++j) {
        const float v = __ldg(a.top_v + o + j);
        const int k = __ldg(a.top_i + o + j);
        if (k < 0) break;
        int q = a.L;
        while (q > 0) {
          const float w = lv[LPR * (q - 1)];
          const int wk = li[LPR * (q - 1)];
          if (wk >= 0 && (w > v || (w == v && wk < k))) break;
          if (q < a.L) {
            lv[LPR * q] = w;
            li[LPR * q] = wk;
          }
          --q;
        }
        if (q == a.L) break;
        lv[LPR * q] = v;
        li[LPR * q] = k;
      }
    }
    __syncwarp();
    draw<LPR>(a.L, lane,
              [&](int j, float &v, int &k) {
                v = lv[LPR * j];
                k = li[LPR * j];
              },
              mv, mine);
  }
  if (WPR > 1) {
    sh.v[warp][lane] = mv;
    sh.k[warp][lane] = mine;
    __syncthreads();
    if (warp == 0)
      draw<LPR>(a.L, lane,
                [&](int j, float &v, int &k) {
                  k = -1;
                  if (lane < WPR) {
                    v = sh.v[lane][j];
                    k = sh.k[lane][j];
                  }
                },
                mv, mine);
  }
  const unsigned group = LPR == 32 ? 0u : (threadIdx.x & 31) & ~(LPR - 1u);  // first lane of the row's group
  const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << group;
  if (sub == 0) {
    // masked (or NaN) columns are in no list: they follow, lowest index first
    const int found = __popc(__ballot_sync(0xffffffffu, mine >= 0) & mask);
    if (__any_sync(0xffffffffu, found < a.cands)) {
      int next = 0;
      for (int j = 0; j < a.cands; ++j) {
        const bool fill = j >= found;
        for (;;) {
          const bool listed = fill & ((__ballot_sync(0xffffffffu, mine == next) & mask) != 0u);
          if (!__any_sync(0xffffffffu, listed)) break;
          next += listed;
        }
        if (fill && lane == j) mine = next;
        if (fill) ++next;
      }
    }
  }
  if (WPR > 1) {
    if (warp == 0) sh.cand[lane] = mine;
    __syncthreads();
  }
  const T *x = static_cast<const T *>(a.x) + (size_t)r * a.d;
  const T *c = static_cast<const T *>(a.c) + (size_t)b * a.K * a.d;
  const float *bias = a.bias ? a.bias + b * a.K : nullptr;
  double v = (double)kNegInf;
  for (int j = 4 * sub; j < a.cands; j += 4 * WPR) {
    int k[4];
    double e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int src = min(j + i, a.cands - 1);
      k[i] = WPR > 1 ? sh.cand[src] : __shfl_sync(0xffffffffu, mine, src, LPR);
    }
    exact_scores<T, LPR>(x, c, bias, a.scale, k, a.d, a.vec, lane, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (lane == j + i) v = e[i];
      if (WPR > 1 && lane == 0 && j + i < a.cands) sh.exact[j + i] = e[i];
    }
  }
  if (WPR > 1) {
    __syncthreads();
    if (warp != 0) return;
    if (lane < a.cands) v = sh.exact[lane];
  }
  const double rank_v = v == v ? v : (double)kNegInf;
  int rank = 0;
  for (int j = 0; j < a.cands; ++j) {
    const double v2 = __shfl_sync(0xffffffffu, rank_v, j, LPR);
    const int k2 = __shfl_sync(0xffffffffu, mine, j, LPR);
    rank += v2 > rank_v || (v2 == rank_v && k2 < mine);
  }
  if (live && lane < a.cands && rank < a.top) {
    a.top_ids[r * a.top + rank] = mine;
    a.top_logp[r * a.top + rank] = v == (double)kNegInf && s == s ? kNegInf
                                                                  : (float)(v - (double)(none ? kNegInf : m) * M_LN2) -
                                                                        ls * kLn2;
  }
}

// ------------------------------------------------------------------ backward
struct RowGrad {  // one row's coefficients
  float a, l, e, lse2, h;
  int id;
  int pad0, pad1;
};

// Coefficients of every row, and the largest bound of |G| over the rows (float
// bits; positive floats order as integers).
__global__ void __launch_bounds__(256)
    k_row_grads(const int32_t *ids, const float *lse, const float *entropy, const float *dlogp, const float *dlse,
                const float *dent, long long rows, int K, RowGrad *out, unsigned *bound, int *err) {
  pdl_wait();
  const long long r = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  float big = 0.f;
  if (r < rows) {
    RowGrad g = {};
    g.id = ids[r];
    if (g.id >= K) atomicCAS(err, DEV_OK, DEV_BAD_ID);
    if (g.id < 0 || g.id >= K) g.id = -1;
    g.a = dlogp && g.id >= 0 ? dlogp[r] : 0.f;
    g.l = dlse ? dlse[r] : 0.f;
    g.e = dent ? dent[r] : 0.f;
    g.h = dent ? entropy[r] : 0.f;
    const float v = lse[r];
    g.lse2 = v * kLog2e;
    if (v == kNegInf) g.a = g.l = g.e = 0.f;  // every column is masked
    if (g.a == 0.f && g.l == 0.f && g.e == 0.f) g.id = -2;  // G is zero whatever the scores hold
    out[r] = g;
    // |p (log p + H)| <= max(1 / e, log K) <= log K + 1
    big = fabsf(g.a) + fabsf(g.l) + fabsf(g.e) * (logf((float)K) + 1.f);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  if ((threadIdx.x & 31) == 0 && big > 0.f) atomicMax(bound, __float_as_uint(big));
}

// The power of two that brings `bound` to [2^13, 2^14), within [2^-100, 2^100].
__device__ __forceinline__ float grad_scale(unsigned bound) {
  const float b = __uint_as_float(bound);
  if (!(b > 0.f) || !(b < INFINITY)) return 1.f;
  int e = 13 - ilogbf(b);
  e = e < -100 ? -100 : e > 100 ? 100 : e;
  return ldexpf(1.f, e);
}

struct GradArgs {
  float scale2;
  const float *bias;
  const RowGrad *rows;    // of the chunk's first row
  const unsigned *bound;  // NULL: unscaled
  long long nr, row_stride, K, Kp;
  void *g;          // (bn, planes, nr, Kp)
  int planes;
  float *colpart;   // (bn, ceil(nr / 32), Kp) or NULL
  long long nblk;
};

template <typename T, bool BIAS, bool SEG>
struct GradEpi {
  using Args = GradArgs;
  static constexpr bool kSeg = SEG;
  const Args &a;
  const int r, lane;
  BiasTile bt;
  const float *bias = nullptr;
  RowGrad q = {};
  long long row = 0;
  float gs = 1.f;
  T *g = nullptr;
  float *cp = nullptr;

  __device__ GradEpi(const Args &args, int lane_, int r_in_tile, int half, uint8_t *smem)
      : a(args), r(r_in_tile), lane(lane_) {
    bt.sb = reinterpret_cast<float *>(smem) + (half * 4 + r_in_tile / 32) * BiasTile::kFloats;
    if (args.bound) gs = grad_scale(*args.bound);
  }
  __device__ void begin(const Unit &w, long long row0) {
    row = row0 + r;
    q = RowGrad{};
    q.id = -2;
    if (row < a.nr) q = a.rows[w.b * a.row_stride + row];
    if (BIAS) bias = a.bias + w.b * a.K;
    g = static_cast<T *>(a.g) + ((size_t)w.b * a.planes * a.nr + row) * a.Kp;
    const long long blk = (row0 + (r & ~31)) >> 5;
    cp = a.colpart && blk < a.nblk ? a.colpart + (w.b * a.nblk + blk) * a.Kp : nullptr;
  }
  static size_t smem_bytes() { return BIAS ? tile::kEpiWarps * BiasTile::kFloats * 4 : 0; }
  __device__ __forceinline__ void prepare(long long col0) {
    if (BIAS) bt.load(bias, col0, a.K, lane);
  }
  __device__ __forceinline__ bool skip(long long col) const { return col >= a.Kp; }
  __device__ __forceinline__ void chunk(const float (&acc)[32], long long col, int i) {
    {
      float v[32];
      scores32<BIAS>(acc, a.scale2, bt, i, col, a.K, v);
      const int rel = q.id - (int)col;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float lp2 = v[j] - q.lse2;
        const float p = ex2(lp2);
        float y = p * (q.l - q.a - q.e * fmaf(fmaxf(lp2, kLowest), kLn2, q.h));
        if (rel == j) y += q.a;
        v[j] = q.id == -2 || v[j] == kNegInf ? 0.f : y;
      }
      if (cp) {
        // column sums of the warp's 32 rows: each exchange halves the columns
        // a lane still carries; lane j ends with column j
        float w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = v[j];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int j = 0; j < o; ++j) {
            const float keep = up ? w[j + o] : w[j], give = up ? w[j] : w[j + o];
            w[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        if (col + lane < a.Kp) cp[col + lane] = w[0];
      }
      if (row < a.nr) {
        if (gs != 1.f) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= gs;
        }
        for (int pl = 0; pl < a.planes; ++pl) {
          uint4 *dst = reinterpret_cast<uint4 *>(g + (size_t)pl * a.nr * a.Kp + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            T h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              h[j] = from_f<T>(v[8 * i + j]);
              v[8 * i + j] -= to_f(h[j]);  // the next plane's value
            }
            if (col + 8 * i < a.Kp) dst[i] = *reinterpret_cast<uint4 *>(h);
          }
        }
      }
    }
  }
  __device__ void end(const Unit &) {}
};

// Plain store of a product: out = alpha * acc, to the result's type or as an
// fp32 partial sum of one part of the contraction.
struct StoreArgs {
  float alpha;
  const unsigned *bound;  // undo the scale of G; NULL: none
  long long rows, cols, pitch;
  void *out;              // (B, rows, cols) with its own row pitch and batch stride
  long long batch_stride;
  float *part;            // (ksplits, B, rows, cols) or NULL
  long long slot;         // elements of one (B, rows, cols) slot
  int add;                // partial sums add to what an earlier block of rows left
};

template <typename T>
__device__ __forceinline__ void store8(T *dst, const float (&v)[8], long long left, bool vec) {
  if (vec && left >= 8) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      T h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = from_f<T>(v[j]);
      *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(h);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) dst[j] = from_f<T>(v[j]);
  }
}

template <typename T, bool SEG>
struct StoreEpi {
  using Args = StoreArgs;
  static constexpr bool kSeg = SEG;
  const Args &a;
  const int r;
  float alpha;
  long long row = 0;
  T *out = nullptr;
  float *part = nullptr;
  bool vec_t, vec_f;

  __device__ StoreEpi(const Args &args, int, int r_in_tile, int, uint8_t *) : a(args), r(r_in_tile) {
    alpha = args.alpha;
    if (args.bound) alpha /= grad_scale(*args.bound);
    vec_t = (args.pitch * sizeof(T)) % 16 == 0;
    vec_f = args.cols % 4 == 0;
  }
  __device__ void begin(const Unit &w, long long row0) {
    row = row0 + r;
    out = static_cast<T *>(a.out) + w.b * a.batch_stride + row * a.pitch;
    if (a.part) part = a.part + w.ks * a.slot + (w.b * a.rows + row) * a.cols;
  }
  __device__ __forceinline__ void prepare(long long) {}
  __device__ __forceinline__ bool skip(long long col) const { return col >= a.cols; }
  __device__ __forceinline__ void chunk(const float (&acc)[32], long long col, int) {
    if (row >= a.rows) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long left = a.cols - col - 8 * i;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[8 * i + j] * alpha;
      if (!a.part) {
        store8<T>(out + col + 8 * i, v, left, vec_t);
      } else {
        float *dst = part + col + 8 * i;
        if (a.add) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) v[j] += dst[j];
        }
        store8<float>(dst, v, left, vec_f);
      }
    }
  }
  __device__ void end(const Unit &) {}
};

// out = the sum of the parts, in order.
template <typename T>
__global__ void __launch_bounds__(256)
    k_sum_parts(const float *part, int parts, long long slot, long long rows, long long cols, long long rows_per_b,
                T *out, long long pitch, long long batch_stride) {
  pdl_wait();
  const long long n = rows * cols;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += part[p * slot + i];
    const long long row = i / cols, b = row / rows_per_b;
    out[b * batch_stride + (row - b * rows_per_b) * pitch + (i - row * cols)] = from_f<T>(s);
  }
}

// dbias[b][k] (+)= the sum of the row blocks' column sums, in a fixed order.
__global__ void __launch_bounds__(256)
    k_sum_cols(const float *colpart, long long nblk, long long Kp, long long K, float *dbias, int add) {
  __shared__ float sm[8][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long long k = (long long)blockIdx.x * 32 + lane;
  const float *src = colpart + (size_t)blockIdx.y * nblk * Kp;
  float s = 0.f;
  if (k < K)
    for (long long j = y; j < nblk; j += 8) s += src[j * Kp + k];
  sm[y][lane] = s;
  __syncthreads();
  if (y == 0 && k < K) {
    for (int j = 1; j < 8; ++j) s += sm[j][lane];
    float *o = dbias + (size_t)blockIdx.y * K + k;
    *o = add ? *o + s : s;
  }
}

// Operand copies: 16-bit rows as they are, fp32 rows as three bf16 planes of
// dp >= d elements (zero padded).  drop: rows whose gradient is zero whatever
// they hold (padding), or table rows that a bias of -inf masks, become zero,
// so that what they hold (NaN included) stays out of the products.
template <typename T>
__global__ void __launch_bounds__(256)
    k_operand(const T *src, long long rows, long long rows_per_b, int d, int dp, const RowGrad *grads,
              const float *bias, void *dst) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const bool drop = (grads && grads[r].id == -2) || (bias && bias[r] == kNegInf);
  const T *in = src + (size_t)r * d;
  if constexpr (sizeof(T) == 2) {
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(dst) + (size_t)r * d);
    for (int j = lane; j < d / 8; j += 32)
      out[j] = drop ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4 *>(in) + j);
  } else {
    const long long b = r / rows_per_b;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(dst) + ((size_t)(b * 3) * rows_per_b + (r - b * rows_per_b)) * dp;
    const size_t plane = (size_t)rows_per_b * dp;
    for (int j = lane; j < dp; j += 32) {
      float v = j < d && !drop ? in[j] : 0.f;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        out[p * plane + j] = h;
        // an infinity (or an overflow of the rounding) leaves no remainder
        const float rest = v - __bfloat162float(h);
        v = fabsf(__bfloat162float(h)) < INFINITY ? rest : 0.f;
      }
    }
  }
}

// ------------------------------------------------------------------ host side
struct Dims {
  int B;
  long long N;
  int K, d, dtype;
  int planes, pairs, dp;
  long long Kp;
};

Dims dims_of(const fk_shape &sh) {
  Dims m;
  m.B = sh.B, m.N = sh.N, m.K = sh.K, m.d = sh.d, m.dtype = sh.dtype;
  m.planes = sh.dtype == FK_F32 ? 3 : 1;
  m.pairs = sh.dtype == FK_F32 ? 6 : 1;
  m.dp = (sh.d + 7) / 8 * 8;
  m.Kp = ((long long)sh.K + 63) / 64 * 64;
  return m;
}

int check_soft(const fk_shape *shape, float scale) {
  if (!shape) return set_error(FK_EINVAL, "shape is NULL");
  if (shape->N < 0) return set_error(FK_EINVAL, "N must be >= 0");
  // the table may be longer than the rows are many
  const long long n = shape->N > shape->K ? shape->N : shape->K;
  FK_TRY(check_shape(shape->B, n, shape->K, shape->d, shape->dtype));
  if (shape->d > (1 << 20)) return set_error(FK_EUNSUPPORTED, "d above 2^20");
  if (!(scale > 0.f) || !(scale < INFINITY)) return set_error(FK_EINVAL, "scale must be positive and finite");
  return FK_OK;
}

long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// Row tiles x column runs over the workers: the fewest rounds of units, with
// the start and the partial results of a unit counted as a quarter of a tile.
Plan plan_runs(int B, long long rows, long long cols, int kdim, int pairs, int planes, int row_bytes) {
  Plan p = {};
  p.cg = group_of(rows);
  const int workers = num_sms() / p.cg;
  p.row_tiles = (int)cdiv(rows, tile::kRows * p.cg);
  p.col_tiles = (int)cdiv(cols, tile::kCols);
  p.kblocks = (int)cdiv(kdim, tile::kK);
  p.pairs = pairs;
  p.planes = planes;
  p.ksplits = 1;
  double best = 1e30;
  p.runs = 1;
  for (int runs = 1; runs <= p.col_tiles && runs <= 2 * workers; ++runs) {
    const double t = (double)cdiv((long long)B * p.row_tiles * runs, workers) * (cdiv(p.col_tiles, runs) + 0.25);
    if (t < best * 0.999) {
      best = t;
      p.runs = runs;
    }
  }
  // rows of one group: 32 MB of the row operand at most, so that they stay in L2
  const long long g = (32LL << 20) / ((long long)tile::kRows * p.cg * row_bytes);
  p.group = (int)std::max(1LL, std::min<long long>(g, p.row_tiles));
  p.units = (int)((long long)B * p.row_tiles * p.runs);
  return p;
}

// One tile per unit, the contraction split so that the last round is not
// mostly idle; a split costs about eight K-blocks (its partial sums).
Plan plan_splits(int B, long long rows, long long cols, long long kdim, int pairs, int planes) {
  Plan p = {};
  p.cg = group_of(rows);
  const int workers = num_sms() / p.cg;
  p.row_tiles = (int)cdiv(rows, tile::kRows * p.cg);
  p.col_tiles = (int)cdiv(cols, tile::kCols);
  p.runs = p.col_tiles;
  p.kblocks = (int)cdiv(kdim, tile::kK);
  p.pairs = pairs;
  p.planes = planes;
  const long long kt = (long long)p.pairs * p.kblocks;
  double best = 1e30;
  p.ksplits = 1;
  for (int ks = 1; ks <= 16 && ks <= kt; ++ks) {
    const double t = (double)cdiv((long long)B * p.row_tiles * p.runs * ks, workers) *
                     ((double)cdiv(kt, ks) + 4.0 + (ks > 1 ? 8.0 : 0.0));
    if (t < best * 0.98) {
      best = t;
      p.ksplits = ks;
    }
  }
  p.group = std::max(1, std::min(p.row_tiles, 16 / p.cg));
  p.units = (int)((long long)B * p.row_tiles * p.runs * p.ksplits);
  return p;
}

bool too_many(const Plan &p, int B) {
  return (double)B * p.row_tiles * p.runs * p.ksplits > 2e9;
}

template <int kCG, class Epi, bool A_MN, bool B_MN>
int launch_group(const CUtensorMap &ta, const CUtensorMap &tb, Plan p, const typename Epi::Args &ea, size_t epi_smem,
                 int ab_fmt, int *err, cudaStream_t s) {
  auto kern = tile::k_tiles<kCG, A_MN, B_MN, Epi>;
  constexpr uint32_t stage = tile::Geo<kCG>::kStageBytes;
  const size_t cap = 227 * 1024 - 1024 - tile::kCtrlBytes;
  p.stages = (int)std::min<size_t>(tile::kMaxStages, (cap - epi_smem) / stage);
  
  p.idesc = sm100::idesc_f32acc((uint32_t)ab_fmt, tile::kRows * kCG, tile::kCols) | (A_MN ? 1u << 15 : 0u) |
            (B_MN ? 1u << 16 : 0u);
  const int smem = (int)(1024 + p.stages * stage + tile::kCtrlBytes + epi_smem);
  FK_TRY(set_smem_limit((const void *)kern, 227 * 1024));
  const int workers = std::min(num_sms() / kCG, p.units);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(workers * kCG);
  cfg.blockDim = dim3(tile::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCG > 1 ? 2 : 1;
  FK_CUDA(cudaLaunchKernelEx(&cfg, kern, ta, tb, p, ea, err));
  return launched();
}

template <class Epi, bool A_MN, bool B_MN>
int launch_tiles(const CUtensorMap &ta, const CUtensorMap &tb, const Plan &p, const typename Epi::Args &ea,
                 size_t epi_smem, int ab_fmt, int *err, cudaStream_t s) {
  if (p.cg == 1) return launch_group<1, Epi, A_MN, B_MN>(ta, tb, p, ea, epi_smem, ab_fmt, err, s);
  return launch_group<2, Epi, A_MN, B_MN>(ta, tb, p, ea, epi_smem, ab_fmt, err, s);
}

// Tensor map of 16-bit elements: (inner, rows, depth) with the row pitch and
// depth stride in elements.
int map_16(CUtensorMap *m, const void *base, bool bf16, long long inner, long long rows, long long depth,
           long long pitch, long long stride, int box_inner, int box_rows) {
  return encode_tiles(m, base, bf16 ? FK_BF16 : FK_F16, inner, rows, depth, pitch, stride, box_inner, box_rows);
}

struct Carve {
  char *base;
  size_t off = 0;
  explicit Carve(void *p) : base(static_cast<char *>(p)) {}
  void *take(size_t bytes) {
    void *r = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return r;
  }
};

// Columns a partial list keeps: at least kSpare more than asked for, 8 or 16 in
// registers, else 32 in shared memory.
int list_length(int top) { return top == 0 ? 0 : top + kSpare <= 8 ? 8 : top + kSpare <= 16 ? 16 : 32; }

struct FwdSpace {
  Plan p;
  int L;
  void *xs, *cs;
  float4 *part;
  float *top_v;
  int32_t *top_i;
  size_t bytes;
};

FwdSpace fwd_space(const Dims &m, int top, void *base) {
  FwdSpace f = {};
  f.p = plan_runs(m.B, m.N, m.K, m.d, m.pairs, m.planes, m.dp * 2 * m.planes);
  f.L = list_length(top);
  Carve w(base);
  const long long parts = 2LL * f.p.runs;
  f.part = (float4 *)w.take((size_t)m.B * m.N * parts * sizeof(float4));
  if (f.L) {
    f.top_v = (float *)w.take((size_t)m.B * m.N * parts * f.L * 4);
    f.top_i = (int32_t *)w.take((size_t)m.B * m.N * parts * f.L * 4);
  }
  if (m.planes == 3) {
    f.xs = w.take((size_t)m.B * 3 * m.N * m.dp * 2);
    f.cs = w.take((size_t)m.B * 3 * m.K * m.dp * 2);
  }
  f.bytes = w.off;
  return f;
}

template <typename T>
int launch_operand(const void *src, long long rows, long long rows_per_b, int d, int dp, const RowGrad *g,
                   const float *bias, void *dst, cudaStream_t s) {
  FK_CUDA(launch_pdl(k_operand<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const T *>(src), rows,
                     rows_per_b, d, dp, g, bias, dst));
  return launched();
}

int operand(const void *src, int dtype, long long rows, long long rows_per_b, int d, int dp, const RowGrad *g,
            const float *bias, void *dst, cudaStream_t s) {
  if (dtype == FK_F32) return launch_operand<float>(src, rows, rows_per_b, d, dp, g, bias, dst, s);
  return launch_operand<__half>(src, rows, rows_per_b, d, dp, g, bias, dst, s);  // 16-bit rows are copied as bits
}

template <class Epi>
int stats_as(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
             cudaStream_t s) {
  return launch_tiles<Epi, false, false>(tx, tc, f.p, a, Epi::smem_bytes(f.L), fmt, err, s);
}

template <bool BIAS, bool SEG>
int stats_seg(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
              cudaStream_t s) {
  if (f.L == 0) return stats_as<StatEpi<BIAS, false, 0, SEG>>(tx, tc, f, a, fmt, err, s);
  if (f.L == 8) return stats_as<StatEpi<BIAS, true, 8, SEG>>(tx, tc, f, a, fmt, err, s);
  if (f.L == 16) return stats_as<StatEpi<BIAS, true, 16, SEG>>(tx, tc, f, a, fmt, err, s);
  return stats_as<StatEpi<BIAS, true, 0, SEG>>(tx, tc, f, a, fmt, err, s);
}

template <bool BIAS>
int scores_stats(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
                 cudaStream_t s) {
  if (f.p.kblocks * f.p.pairs > tile::kSegBlocks) return stats_seg<BIAS, true>(tx, tc, f, a, fmt, err, s);
  return stats_seg<BIAS, false>(tx, tc, f, a, fmt, err, s);
}

template <typename T, int LPR, int WPR>
int launch_join_as(const JoinArgs &j, cudaStream_t s) {
  const int per_block = WPR > 1 ? 1 : kJoinWarps * (32 / LPR);
  const size_t smem = j.parts > LPR * WPR ? (size_t)kJoinWarps * 64 * j.L * 4 : 0;
  if (smem) FK_TRY(set_smem_limit((const void *)k_join<T, LPR, WPR>, kJoinWarps * 64 * 32 * 4));
  FK_CUDA(launch_pdl(k_join<T, LPR, WPR>, dim3((unsigned)cdiv(j.rows, per_block)), dim3(32 * kJoinWarps), smem, s, j));
  return launched();
}

// Eight lanes hold eight candidates at most; a block per row pays while the
// rows alone do not fill the SMs.
template <typename T>
int launch_join(const JoinArgs &j, cudaStream_t s) {
  if (j.L && j.rows <= 4096) return launch_join_as<T, 32, 8>(j, s);
  if (j.L <= 8 && j.parts <= 64) return launch_join_as<T, 8, 1>(j, s);
  return launch_join_as<T, 32, 1>(j, s);
}

struct BwdSpace {
  Plan pg, px, pw;      // of a full block of rows
  int bn;               // batches per block
  long long nr;         // rows per block
  unsigned *bound;
  RowGrad *rows;
  void *xs, *cs, *g;    // operand copies; cs NULL where c itself is read
  float *colpart, *partx, *partw;
  bool w_parts;         // dc goes through fp32 partial sums
  size_t bytes;
};

constexpr long long kGradBudget = 4LL << 30;  // bytes of G held at a time

BwdSpace bwd_space(const Dims &m, bool bias, bool dbias, void *base) {
  BwdSpace f = {};
  const long long row_bytes = m.Kp * 2 * m.planes;
  f.nr = std::min<long long>(m.N, std::max<long long>(256, kGradBudget / row_bytes / 256 * 256));
  f.bn = f.nr < m.N ? 1 : (int)std::max<long long>(1, std::min<long long>(m.B, kGradBudget / (row_bytes * f.nr)));
  f.pg = plan_runs(f.bn, f.nr, m.Kp, m.d, m.pairs, m.planes, m.dp * 2 * m.planes);
  f.px = plan_splits(f.bn, f.nr, m.d, m.K, m.pairs, m.planes);
  f.pw = plan_splits(f.bn, m.K, m.d, f.nr, m.pairs, m.planes);
  f.w_parts = f.pw.ksplits > 1 || f.nr < m.N;
  Carve w(base);
  f.bound = (unsigned *)w.take(16);
  f.rows = (RowGrad *)w.take((size_t)m.B * m.N * sizeof(RowGrad));
  f.xs = w.take((size_t)m.B * m.planes * m.N * m.dp * 2);
  if (m.planes == 3 || bias) f.cs = w.take((size_t)m.B * m.planes * m.K * m.dp * 2);
  f.g = w.take((size_t)f.bn * f.nr * row_bytes);
  if (dbias) f.colpart = (float *)w.take((size_t)f.bn * cdiv(f.nr, 32) * m.Kp * 4);
  if (f.px.ksplits > 1) f.partx = (float *)w.take((size_t)f.px.ksplits * f.bn * f.nr * m.d * 4);
  if (f.w_parts) f.partw = (float *)w.take((size_t)f.pw.ksplits * f.bn * m.K * m.d * 4);
  f.bytes = w.off;
  return f;
}

template <typename T>
int launch_sum_parts(const float *part, const Plan &p, int B, long long rows, long long cols, void *out,
                     long long pitch, long long batch_stride, cudaStream_t s) {
  const long long n = (long long)B * rows * cols;
  const long long blocks = std::min<long long>(cdiv(n, 256), (long long)num_sms() * 16);
  FK_CUDA(launch_pdl(k_sum_parts<T>, dim3((unsigned)blocks), dim3(256), 0, s, part, p.ksplits, n, (long long)B * rows,
                     cols, rows, static_cast<T *>(out), pitch, batch_stride));
  return launched();
}

// T: the gradients' type; G: the 16-bit type of the products' operands.
template <typename T, typename G, bool BIAS>
int backward_typed(const Dims &m, const BwdSpace &f, const void *xo, const void *co, const void *cmul, const float *bias,
                   float scale, void *dx, void *dc, float *dbias, int *err, cudaStream_t s) {
  const bool bf = m.dtype != FK_F16;
  const int fmt = bf ? 1 : 0;
  const size_t es = esize(m.dtype);
  const unsigned *bound = m.dtype == FK_F16 ? f.bound : nullptr;
  for (int b0 = 0; b0 < m.B; b0 += f.bn) {
    const int bn = std::min(f.bn, m.B - b0);
    for (long long r0 = 0; r0 < m.N; r0 += f.nr) {
      const long long nr = std::min(f.nr, m.N - r0);
      const size_t xoff = ((size_t)b0 * m.planes * m.N + r0) * m.dp * 2, coff = (size_t)b0 * m.planes * m.K * m.dp * 2;
      // scores again, and from them G
      Plan pg = f.pg;
      if (bn != f.bn || nr != f.nr) pg = plan_runs(bn, nr, m.Kp, m.d, m.pairs, m.planes, m.dp * 2 * m.planes);
      CUtensorMap tx, tc;
      FK_TRY(map_16(&tx, (const char *)xo + xoff, bf, m.dp, nr, (long long)bn * m.planes, m.dp, m.N * m.dp, tile::kK,
                    tile::kRows));
      FK_TRY(map_16(&tc, (const char *)co + coff, bf, m.dp, m.K, (long long)bn * m.planes, m.dp, (long long)m.K * m.dp,
                    tile::kK, tile::kCols / pg.cg));
      GradArgs ga = {};
      ga.scale2 = scale * kLog2e;
      ga.bias = bias ? bias + (size_t)b0 * m.K : nullptr;
      ga.rows = f.rows + (size_t)b0 * m.N + r0;
      ga.bound = bound;
      ga.nr = nr, ga.row_stride = m.N, ga.K = m.K, ga.Kp = m.Kp;
      ga.g = f.g;
      ga.planes = m.planes;
      ga.colpart = dbias ? f.colpart : nullptr;
      ga.nblk = cdiv(nr, 32);
      // scores as exact as the forward pass's where fp32 results hang on them;
      // a 16-bit gradient does not show the difference (2^-15 against 2^-9)
      if ((m.planes == 3 || dbias) && pg.kblocks * pg.pairs > tile::kSegBlocks)
        FK_TRY((launch_tiles<GradEpi<G, BIAS, true>, false, false>(tx, tc, pg, ga, GradEpi<G, BIAS, true>::smem_bytes(), fmt, err, s)));
      else
        FK_TRY((launch_tiles<GradEpi<G, BIAS, false>, false, false>(tx, tc, pg, ga, GradEpi<G, BIAS, false>::smem_bytes(), fmt, err, s)));
      if (dbias) {
        FK_CUDA(launch_pdl(k_sum_cols, dim3((unsigned)cdiv(m.K, 32), bn), dim3(256), 0, s, (const float *)f.colpart,
                           ga.nblk, m.Kp, (long long)m.K, dbias + (size_t)b0 * m.K, r0 > 0 ? 1 : 0));
        FK_TRY(launched());
      }
      // dx = G C: the contraction is the table's rows
      if (dx) {
        CUtensorMap tg, tcm;
        FK_TRY(map_16(&tg, f.g, bf, m.Kp, nr, (long long)bn * m.planes, m.Kp, nr * m.Kp, tile::kK, tile::kRows));
        FK_TRY(map_16(&tcm, (const char *)cmul + coff, bf, m.dp, m.K, (long long)bn * m.planes, m.dp,
                      (long long)m.K * m.dp, 64, tile::kK));
        Plan px = f.px;
        if (bn != f.bn || nr != f.nr) {
          px = plan_splits(bn, nr, m.d, m.K, m.pairs, m.planes);
          if (px.ksplits > f.px.ksplits || (long long)px.ksplits * bn * nr > (long long)f.px.ksplits * f.bn * f.nr) {
            px.ksplits = f.px.ksplits;
            px.units = (int)((long long)bn * px.row_tiles * px.runs * px.ksplits);
          }
        }
        StoreArgs sa = {};
        sa.alpha = scale;
        sa.bound = bound;
        sa.rows = nr, sa.cols = m.d, sa.pitch = m.d;
        sa.out = (char *)dx + ((size_t)b0 * m.N + r0) * m.d * es;
        sa.batch_stride = m.N * m.d;
        sa.part = px.ksplits > 1 ? f.partx : nullptr;
        sa.slot = (long long)bn * nr * m.d;
        FK_TRY((launch_tiles<StoreEpi<T, sizeof(T) == 4>, false, true>(tg, tcm, px, sa, 0, fmt, err, s)));
        if (sa.part)
          FK_TRY(launch_sum_parts<T>(f.partx, px, bn, nr, m.d, sa.out, m.d, sa.batch_stride, s));
      }
      // dc = G^T X: the contraction is the rows
      if (dc) {
        CUtensorMap tg, txm;
        FK_TRY(map_16(&tg, f.g, bf, m.Kp, nr, (long long)bn * m.planes, m.Kp, nr * m.Kp, 64, tile::kK));
        FK_TRY(map_16(&txm, (const char *)f.xs + xoff, bf, m.dp, nr, (long long)bn * m.planes, m.dp, m.N * m.dp, 64,
                      tile::kK));
        Plan pw = f.pw;
        if (bn != f.bn || nr != f.nr) {
          // the partial sums keep their slots over all blocks of rows
          pw = plan_splits(bn, m.K, m.d, nr, m.pairs, m.planes);
          const long long kt = (long long)pw.pairs * pw.kblocks;
          pw.ksplits = (int)std::min<long long>(f.pw.ksplits, kt);
          pw.units = (int)((long long)bn * pw.row_tiles * pw.runs * pw.ksplits);
        }
        StoreArgs sa = {};
        sa.alpha = scale;
        sa.bound = bound;
        sa.rows = m.K, sa.cols = m.d, sa.pitch = m.d;
        sa.out = (char *)dc + (size_t)b0 * m.K * m.d * es;
        sa.batch_stride = (long long)m.K * m.d;
        sa.part = f.w_parts ? f.partw : nullptr;
        sa.slot = (long long)bn * m.K * m.d;
        sa.add = r0 > 0;
        FK_TRY((launch_tiles<StoreEpi<T, sizeof(T) == 4>, true, true>(tg, txm, pw, sa, 0, fmt, err, s)));
        if (sa.part && r0 + nr >= m.N) {
          Plan all = f.pw;
          all.ksplits = f.nr < m.N ? f.pw.ksplits : pw.ksplits;
          FK_TRY(launch_sum_parts<T>(f.partw, all, bn, m.K, m.d, sa.out, m.d, sa.batch_stride, s));
        }
      }
    }
  }
  return FK_OK;
}

template <typename T, typename G>
int backward_bias(const Dims &m, const BwdSpace &f, const void *xo, const void *co, const void *cmul, const float *bias,
                  float scale, void *dx, void *dc, float *dbias, int *err, cudaStream_t s) {
  if (bias) return backward_typed<T, G, true>(m, f, xo, co, cmul, bias, scale, dx, dc, dbias, err, s);
  return backward_typed<T, G, false>(m, f, xo, co, cmul, bias, scale, dx, dc, dbias, err, s);
}

}  // namespace
}  // namespace fk

using namespace fk;

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
               float *logp, float *lse, float *entropy, int top, int32_t *top_ids, float *top_logp, void *workspace,
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
    FK_TRY(operand(x, m.dtype, m.B * m.N, m.N, m.d, m.dp, nullptr, nullptr, f.xs, s));
    FK_TRY(operand(c, m.dtype, (long long)m.B * m.K, m.K, m.d, m.dp, nullptr, nullptr, f.cs, s));
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
  a.parts = 2 * f.p.runs;
  a.L = f.L;
  a.part = f.part, a.top_v = f.top_v, a.top_i = f.top_i;
  if (bias) FK_TRY(scores_stats<true>(tx, tc, f, a, bf ? 1 : 0, err, s));
  else FK_TRY(scores_stats<false>(tx, tc, f, a, bf ? 1 : 0, err, s));
  JoinArgs j = {};
  j.part = f.part, j.top_v = f.top_v, j.top_i = f.top_i;
  j.ids = ids, j.x = x, j.c = c, j.bias = bias, j.scale = scale;
  j.rows = m.B * m.N, j.N = m.N, j.K = m.K, j.d = m.d;
  j.parts = a.parts, j.L = f.L, j.cands = std::min(f.L, m.K), j.top = top;
  j.logp = logp, j.lse = lse, j.entropy = entropy, j.top_logp = top_logp, j.top_ids = top_ids;
  j.err = err;
  j.vec = m.d * esize(m.dtype) % 16 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(c)) & 15) == 0;
  if (m.dtype == FK_F32) return launch_join<float>(j, s);
  if (m.dtype == FK_BF16) return launch_join<__nv_bfloat16>(j, s);
  return launch_join<__half>(j, s);
}

int fk_logprob_backward_workspace(const fk_shape *shape, int with_bias, int with_dbias, long long *bytes) {
  FK_TRY(check_soft(shape, 1.f));
  if (!bytes) return set_error(FK_EINVAL, "bytes is NULL");
  const BwdSpace f = bwd_space(dims_of(*shape), with_bias != 0, with_dbias != 0, nullptr);
  if (too_many(f.pg, f.bn) || too_many(f.px, f.bn) || too_many(f.pw, f.bn))
    return set_error(FK_EUNSUPPORTED, "too many tiles");
  *bytes = (long long)f.bytes;
  return FK_OK;
}

int fk_logprob_backward(const fk_shape *shape, const void *x, const void *c, const float *bias, float scale,
                        const int32_t *ids, const float *lse, const float *entropy, const float *dlogp,
                        const float *dlse, const float *dentropy, void *dx, void *dc, float *dbias, void *workspace,
                        long long workspace_bytes, fk_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FK_TRY(check_soft(shape, scale));
  if (dbias && !bias) return set_error(FK_EINVAL, "dbias without bias");
  long long need = 0;
  FK_TRY(fk_logprob_backward_workspace(shape, bias != nullptr, dbias != nullptr, &need));
  const Dims m = dims_of(*shape);
  const bool al = m.dtype != FK_F32;
  FK_TRY(check_ptr(c, "c", al));
  if (dc) {
    FK_TRY(check_ptr(dc, "dc", true));
    FK_TRY(check_dev(dc, "dc"));
  }
  FK_TRY(check_dev_opt(dbias, "dbias"));
  if (m.N == 0) {  // no rows: the table's gradients are zero
    if (dc) FK_CUDA(cudaMemsetAsync(dc, 0, (size_t)m.B * m.K * m.d * esize(m.dtype), s));
    if (dbias) FK_CUDA(cudaMemsetAsync(dbias, 0, (size_t)m.B * m.K * 4, s));
    return FK_OK;
  }
  FK_TRY(check_ptr(x, "x", al));
  FK_TRY(check_ptr(ids, "ids", false));
  FK_TRY(check_ptr(lse, "lse", false));
  if (dentropy) FK_TRY(check_ptr(entropy, "entropy", false));
  if (dx) {
    FK_TRY(check_ptr(dx, "dx", true));
    FK_TRY(check_dev(dx, "dx"));
  }
  FK_TRY(check_ptr(workspace, "workspace", true));
  if (workspace_bytes < need)
    return set_error(FK_EINVAL, "workspace is smaller than fk_logprob_backward_workspace asks for");
  FK_TRY(check_dev(x, "x"));
  FK_TRY(check_dev(c, "c"));
  FK_TRY(check_dev_opt(bias, "bias"));
  FK_TRY(check_dev(ids, "ids"));
  FK_TRY(check_dev(lse, "lse"));
  FK_TRY(check_dev_opt(entropy, "entropy"));
  FK_TRY(check_dev_opt(dlogp, "dlogp"));
  FK_TRY(check_dev_opt(dlse, "dlse"));
  FK_TRY(check_dev_opt(dentropy, "dentropy"));
  FK_TRY(check_dev(workspace, "workspace"));
  if (!dx && !dc && !dbias) return FK_OK;
  int *err = nullptr;
  FK_TRY(soft_error_word(&err));
  const BwdSpace f = bwd_space(m, bias != nullptr, dbias != nullptr, workspace);
  const long long rows = m.B * m.N;
  FK_CUDA(cudaMemsetAsync(f.bound, 0, 16, s));
  k_row_grads<<<(unsigned)cdiv(rows, 256), 256, 0, s>>>(ids, lse, entropy, dlogp, dlse, dentropy, rows, m.K, f.rows,
                                                        f.bound, err);
  FK_TRY(launched());
  FK_CUDA(cudaGetLastError());
  FK_TRY(operand(x, m.dtype, rows, m.N, m.d, m.dp, f.rows, nullptr, f.xs, s));
  if (f.cs) FK_TRY(operand(c, m.dtype, (long long)m.B * m.K, m.K, m.d, m.dp, nullptr, bias, f.cs, s));
  // a dropped row's or column's scores do not count (its G is zero), so the
  // recomputed scores may read the cleaned copies as well
  const void *co = f.cs ? f.cs : c;
  if (m.dtype == FK_F32)
    return backward_bias<float, __nv_bfloat16>(m, f, f.xs, co, co, bias, scale, dx, dc, dbias, err, s);
  if (m.dtype == FK_BF16)
    return backward_bias<__nv_bfloat16, __nv_bfloat16>(m, f, f.xs, co, co, bias, scale, dx, dc, dbias, err, s);
  return backward_bias<__half, __half>(m, f, f.xs, co, co, bias, scale, dx, dc, dbias, err, s);
}

}  // extern "C"
