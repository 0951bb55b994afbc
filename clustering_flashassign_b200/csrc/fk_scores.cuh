// The forward epilogue of the token log probabilities: running softmax
// statistics and best columns of every row.
#pragma once

#include "fk_logprob.cuh"

namespace fk {
namespace soft {

// Running statistics of one row per thread.
//
// The sums refer to a whole number m that follows the row's maximum with a slack
// of 2: a chunk's exponentials then rarely wait for its maximum, and moving m
// multiplies the sums by a power of two, without a rounding.
//
// The best columns.  Eight columns of which no row of the warp wants anything
// (their maximum beats none of the lists) cost a comparison.  Otherwise they
// are drained from their maximum downwards, every lane inserting its own best
// column in the same step, until no lane's remainder beats its list.  A list of
// 4 to 16 (LREG) sits in registers, where an insertion is a branchless shift of
// five instructions a place; a longer one in shared memory.
template <bool BIAS, bool TOP, int LREG, bool SEG>
struct StatEpi {
  using Args = StatArgs;
  static constexpr int kSeg = SEG ? tile::kSegBlocks : 0;
  static constexpr int kRegs = SEG && TOP ? 160 : 152;
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
    id = row < a.N ? a.ids[at] : -1;
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
  __device__ __forceinline__ void prepare(long long col0, int stride) {
    if (BIAS && !skip(col0)) bt.load(bias, col0, stride, a.K, lane);
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
    const bool some_masked = scores32<BIAS>(acc, a.scale2, bt, i, col, a.K, t);
    float g[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float *v = t + 8 * q;
      g[q] = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
    }
    const float cm = max3(fmaxf(g[0], g[1]), g[2], g[3]);
    const float c2 = BIAS ? cm : __fmul_rn(cm, a.scale2);
    if (c2 > m + 2.f) {  // always the case for the first finite chunk
      const float up = ceilf(c2);
      if (m != kNegInf) {
        const float f = pow2(m - up);
        us = f * fmaf(m - up, sum, us);
        sum *= f;
      }
      m = up;
    }
    const float ms = m == kNegInf ? 0.f : m;
    const float2 ref = make_float2(-ms, -ms), sc = make_float2(a.scale2, a.scale2);
    float2 s2[2] = {}, u2[2] = {};
    const bool coarse = !BIAS && fabsf(ms) >= kCoarse;
    if (!some_masked && !coarse) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 v = make_float2(t[2 * j], t[2 * j + 1]);
        const float2 dd = BIAS ? __fadd2_rn(v, ref) : __ffma2_rn(v, sc, ref);
        const float2 e = make_float2(ex2(dd.x), ex2(dd.y));
        s2[j & 1] = __fadd2_rn(s2[j & 1], e);
        u2[j & 1] = __ffma2_rn(e, dd, u2[j & 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 v = make_float2(t[2 * j], t[2 * j + 1]);
        float2 dd = BIAS ? __fadd2_rn(v, ref) : __ffma2_rn(v, sc, ref);
        if (coarse) dd = make_float2(__fmul_rn(v.x, a.scale2) - ms, __fmul_rn(v.y, a.scale2) - ms);
        const float2 e = make_float2(ex2(dd.x), ex2(dd.y));
        s2[j & 1] = __fadd2_rn(s2[j & 1], e);
        u2[j & 1] = __ffma2_rn(e, make_float2(fmaxf(dd.x, kLowest), fmaxf(dd.y, kLowest)), u2[j & 1]);
      }
    }
    sum += (s2[0].x + s2[1].x) + (s2[0].y + s2[1].y);
    us += (u2[0].x + u2[1].x) + (u2[0].y + u2[1].y);
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
    const long long p = at * a.parts + w.run * 3 + half;
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

template <class Epi>
int stats_as(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
             cudaStream_t s) {
  return launch_tiles<Epi, false, false>(tx, tc, f.p, a, Epi::smem_bytes(f.L), fmt, err, s);
}

template <bool BIAS, bool SEG>
int stats_seg(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
              cudaStream_t s) {
  if (f.L == 0) return stats_as<StatEpi<BIAS, false, 0, SEG>>(tx, tc, f, a, fmt, err, s);
  if (f.L == 4) return stats_as<StatEpi<BIAS, true, 4, SEG>>(tx, tc, f, a, fmt, err, s);
  if (f.L == 8) return stats_as<StatEpi<BIAS, true, 8, SEG>>(tx, tc, f, a, fmt, err, s);
  if (f.L == 12) return stats_as<StatEpi<BIAS, true, 12, SEG>>(tx, tc, f, a, fmt, err, s);
  if (f.L == 16) return stats_as<StatEpi<BIAS, true, 16, SEG>>(tx, tc, f, a, fmt, err, s);
  return stats_as<StatEpi<BIAS, true, 0, SEG>>(tx, tc, f, a, fmt, err, s);
}

template <bool BIAS>
int scores_stats(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
                 cudaStream_t s) {
  if (f.p.kblocks * f.p.pairs > tile::kSegBlocks) return stats_seg<BIAS, true>(tx, tc, f, a, fmt, err, s);
  return stats_seg<BIAS, false>(tx, tc, f, a, fmt, err, s);
}

}  // namespace soft
}  // namespace fk
