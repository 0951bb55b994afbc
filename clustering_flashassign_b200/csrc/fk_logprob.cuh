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
// once to the operands' type (in two parts in small calls; bf16: relative 2^-9 of each value; fp16: 2^-11
// after a power-of-two scale that brings the largest possible |G| of the call
// to 2^14; fp32: three bf16 planes, 2^-25), and multiplies G with C and X.
// G is held for a block of rows at a time, sized by a fixed budget.
// The column sums of dbias use G before the rounding.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fk_tile_engine.cuh"

namespace fk {
namespace soft {

using tile::Plan;
using tile::Unit;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;
// Below 2^-256 of the maximum a term is zero in fp32; where columns are masked
// the clamp keeps 0 * -inf out of the entropy sum (a NaN sum stays NaN).
constexpr float kLowest = -256.f;
// Columns beyond `top` that the running lists keep: the lists rank by fp32
// scores, and the final order is settled in fp64 among top + kSpare columns.
// Which columns are among them rests on the fp32 scores: more than kSpare others
// within the rounding of the top-th may leave one of them out.  (An exact cut
// would be a second product in fp64 for every row of such a table.)
constexpr int kSpare = 2;
constexpr int kMaxTop = 28;
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// CTAs per tile.  Pairs halve the operand traffic per product, which counts when
// the tensor cores are busy: with two rounds of 128 x 256 tiles of some depth
// for all SMs, and more rows than one CTA holds.  Less work is spread over
// single CTAs (N 512, K 1000, d 256: scores 9.1 us against 10.6, dX 11.3
// against 14.4, dC 11.0 against 13.1; dX at N 1777, K 20003, d 1024, 56 deep
// tiles: 69 us against 63 by pairs).
inline int group_of(long long rows, double tiles) { return rows <= tile::kRows || tiles < 2.0 * num_sms() ? 1 : 2; }

// Few tiles of a deep contraction take pairs too, if all find room at once: a
// tile's time is then that of its copies, whose rows the copy unit takes one by
// one, 384 a K-block by one CTA and 256 by a pair (fp32, N 92, K 326, d 3250, 306
// K-blocks: 140 us against 186; at 48 to 64 K-blocks 2 to 4 us slower, since pairs
// start later).
constexpr int kDeepBlocks = 128;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// 2^n of a whole n <= 0 (0 below the normal range), exactly.
__device__ __forceinline__ float pow2(float n) {
  return n >= -126.f ? __int_as_float(((int)n + 127) << 23) : 0.f;
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

// A finite bias beyond 2.3e38 in magnitude counts as that: the lowest values of
// bf16 and fp32, which programs mask with, would overflow times log2 e, and
// 0 * inf is NaN.  From 1e30 on, a column takes the path of masked ones, which
// keeps differences from it finite; it adds exactly nothing beside an ordinary
// column.
constexpr float kMaxBias = 2.3e38f;
constexpr float kMaskBias = 1e30f;
__device__ __forceinline__ float clamp_bias(float b) {
  return fabsf(b) > kMaxBias && fabsf(b) < INFINITY ? copysignf(kMaxBias, b) : b;
}

// A warp's bias of its (at most four) 32-column chunks of a tile, times log2 e,
// in shared memory; columns past the last count as masked.  `masked`: which of
// the chunks hold a masked column, or one with a bias beyond kMaskBias.
struct BiasTile {
  static constexpr int kFloats = 128;
  float *sb;
  unsigned masked = 0;
  __device__ __forceinline__ void load(const float *bias, long long col0, int stride, long long K, int lane) {
    __syncwarp();  // the previous tile's values have been read
    masked = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long col = col0 + i * stride + lane;
      const float b = col < K ? bias[col] : kNegInf;
      sb[i * 32 + lane] = clamp_bias(b) * kLog2e;
      if (__any_sync(0xffffffffu, fabsf(b) > kMaskBias)) masked |= 1u << i;
    }
    __syncwarp();
  }
};

// The 32 scores of a thread's row in columns [col, col + 32), the warp's
// chunk i: in base 2 with a bias, else the products as they are (the scale is
// positive).  A bias of -inf masks its column whatever the product holds, and
// columns past the last are masked; returns whether differences need a clamp.
template <bool BIAS>
__device__ __forceinline__ bool scores32(const float (&r)[32], float scale2, const BiasTile &bt, int i, long long col,
                                         long long K, float (&t)[32]) {
  if (BIAS) {
    const float4 *sb = reinterpret_cast<const float4 *>(bt.sb + i * 32);
    const float2 s2 = make_float2(scale2, scale2);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 b = sb[j];
      const float2 lo = __ffma2_rn(make_float2(r[4 * j], r[4 * j + 1]), s2, make_float2(b.x, b.y));
      const float2 hi = __ffma2_rn(make_float2(r[4 * j + 2], r[4 * j + 3]), s2, make_float2(b.z, b.w));
      t[4 * j] = lo.x, t[4 * j + 1] = lo.y, t[4 * j + 2] = hi.x, t[4 * j + 3] = hi.y;
    }
    const bool some = bt.masked >> i & 1u;
    if (some) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (bt.sb[i * 32 + j] == kNegInf) t[j] = kNegInf;
    }
    return some;
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j] = r[j];
    const bool some = col + 32 > K;
    if (some) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j >= K) t[j] = kNegInf;
    }
    return some;
  }
}

// References from here on are no longer exact to a unit, and the rounding of a
// product times the scale (without a bias it is not rounded before the reference
// is subtracted) would show as a difference from its own maximum, up to 2^128 and
// more in the sum: such products are rounded first, wherever they are used.
constexpr float kCoarse = 8388608.f;

// One row's coefficients: G_k = p (c1 + c2 log2 p) + a 1[k = id], p = 2^(t_k - lse2).
// lse in base 2 is lse2 and a remainder below its rounding; c1 and c2 carry it.
struct RowGrad {
  float a, c1, c2, lse2;
  int id;  // -1: no target, -2: G is zero whatever the scores hold
  int pad0, pad1, pad2;
};

struct StatArgs {
  float scale2;
  const float *bias;  // (B, K) or NULL
  const int32_t *ids;
  long long N, K;
  int parts;  // partial results per row: 3 * runs
  int L;      // columns kept per partial list, 0: none
  float4 *part;          // (B, N, parts): m, sum, sum e (t - m), target score (as scores32 gives it)
  float *top_v;          // (B, N, parts, L)
  int32_t *top_i;
};

// Up to this many rows, a row whose alternatives are asked for gets a block in the join.
constexpr long long kJoinBlockRows = 4096;

struct JoinArgs {
  const float4 *part;
  const float *top_v;
  const int32_t *top_i;
  const int32_t *ids;
  const void *x, *c;
  const float *bias;
  float scale;
  float unit2;  // of the stored scores in base 2: scale * log2 e, with a bias 1
  long long rows, N, K;
  int d, parts, L, cands, top;  // L: length of a partial list; cands = min(K, top + kSpare)
  bool vec;  // rows of x and c can be read 16 bytes at a time
  float *logp, *lse, *lse_rest, *entropy, *top_logp;
  int32_t *top_ids;
  int *err;
  unsigned *max_norm2;  // (B): scratch of the joins without a block per row, or NULL
};

struct Dims {
  int B;
  long long N;
  int K, d, dtype;
  int planes, pairs, dp;
  int g_planes, g_pairs;  // of G, and of its products
  long long Kp;
};

inline Dims dims_of(const fk_shape &sh) {
  Dims m;
  m.B = sh.B, m.N = sh.N, m.K = sh.K, m.d = sh.d, m.dtype = sh.dtype;
  m.planes = sh.dtype == FK_F32 ? 3 : 1;
  m.pairs = sh.dtype == FK_F32 ? 6 : 1;
  // G is rounded once, which for a row or two can show (their gradients may be
  // differences of a few large terms): where it costs nothing to speak of, G is
  // kept in two parts, and the rounding of the result is the only one.  The
  // products of one such call take 10 us at most, or read the table for 64 rows
  // at most.
  const double work = (double)sh.B * sh.N * sh.K * sh.d;
  m.g_planes = m.planes == 3 ? 3 : work <= 2147483648.0 || sh.N <= 64 ? 2 : 1;
  m.g_pairs = m.planes == 3 ? 6 : m.g_planes;
  m.dp = (sh.d + 7) / 8 * 8;
  m.Kp = ((long long)sh.K + 63) / 64 * 64;
  return m;
}

inline int check_soft(const fk_shape *shape, float scale) {
  if (!shape) return set_error(FK_EINVAL, "shape is NULL");
  if (shape->N < 0) return set_error(FK_EINVAL, "N must be >= 0");
  // the table may be longer than the rows are many
  const long long n = shape->N > shape->K ? shape->N : shape->K;
  FK_TRY(check_shape(shape->B, n, shape->K, shape->d, shape->dtype));
  // row numbers of the last tile's empty rows are ints too
  if (shape->N > 0x7fffffffLL - 512) return set_error(FK_EUNSUPPORTED, "N above 2^31 - 513");
  if (shape->d > (1 << 20)) return set_error(FK_EUNSUPPORTED, "d above 2^20");
  if (!(scale > 0.f) || !(scale * kLog2e < INFINITY))
    return set_error(FK_EINVAL, "scale must be positive and finite (below 2.3e38)");
  return FK_OK;
}

// Row tiles x column runs over the workers: the fewest rounds of units, with
// the start and the partial results of a unit counted as a quarter of a tile.
inline Plan plan_runs(int B, long long rows, long long cols, int kdim, int pairs, int planes, int row_bytes) {
  Plan p = {};
  p.cg = group_of(rows, (double)B * cdiv(rows, tile::kRows) * cdiv(cols, tile::kCols));
  p.kblocks = (int)cdiv(kdim, tile::kK);
  if (p.kblocks * pairs >= kDeepBlocks &&
      2.0 * B * cdiv(rows, 2 * tile::kRows) * cdiv(cols, tile::kCols) <= num_sms())
    p.cg = 2;
  const int workers = num_sms() / p.cg;
  p.row_tiles = (int)cdiv(rows, tile::kRows * p.cg);
  p.col_tiles = (int)cdiv(cols, tile::kCols);
  p.pairs = pairs;
  p.planes_a = p.planes_b = planes;
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
inline Plan plan_splits(int B, long long rows, long long cols, long long kdim, int pairs, int planes_a, int planes_b) {
  Plan p = {};
  const double depth = std::max(1.0, pairs * cdiv(kdim, tile::kK) / 16.0);
  p.cg = group_of(rows, (double)B * cdiv(rows, tile::kRows) * cdiv(cols, tile::kCols) * depth);
  const int workers = num_sms() / p.cg;
  p.row_tiles = (int)cdiv(rows, tile::kRows * p.cg);
  p.col_tiles = (int)cdiv(cols, tile::kCols);
  p.runs = p.col_tiles;
  p.kblocks = (int)cdiv(kdim, tile::kK);
  p.pairs = pairs;
  p.planes_a = planes_a;
  p.planes_b = planes_b;
  const long long kt = (long long)p.pairs * p.kblocks;
  double best = 1e30;
  p.ksplits = 1;
  for (int ks = 1; ks <= 64 && ks <= kt; ++ks) {
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

inline bool too_many(const Plan &p, int B) {
  return (double)B * p.row_tiles * p.runs * p.ksplits > 2e9;
}

// The register split waits for registers that the launch must have brought.
int check_registers(const void *kernel, int regs);

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
  FK_TRY(check_registers((const void *)kern, tile::kLaunchRegs));
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
inline int map_16(CUtensorMap *m, const void *base, bool bf16, long long inner, long long rows, long long depth,
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

// Columns a partial list keeps: at least kSpare more than asked for; up to 16
// in registers (an insertion costs five instructions a place), else 32 in
// shared memory.
constexpr int list_length(int top) { return top == 0 ? 0 : top + kSpare <= 16 ? (top + kSpare + 3) / 4 * 4 : 32; }

struct FwdSpace {
  Plan p;
  int L, parts;
  void *xs, *cs;
  float4 *part;
  float *top_v;
  int32_t *top_i;
  unsigned *max_norm2;
  size_t bytes;
};


// One row's operand copy, by a warp: 16-bit rows as they are, fp32 rows as three
// bf16 planes of dp >= d elements (zero padded).  drop: rows whose gradient is
// zero whatever they hold (padding), or table rows that a bias of -inf masks,
// become zero, so that what they hold (NaN included) stays out of the products.
// The kernel before may still have been writing src when this one became
// resident: ordinary loads.
template <typename T>
__device__ __forceinline__ void copy_row(const T *src, long long r, long long rows_per_b, int d, int dp, bool drop,
                                         void *dst, int lane) {
  const T *in = src + (size_t)r * d;
  if constexpr (sizeof(T) == 2) {
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(dst) + (size_t)r * d);
    const uint4 *in16 = reinterpret_cast<const uint4 *>(in);
    constexpr int U = 4;  // loads in flight
    for (int j0 = lane; j0 < d / 8; j0 += 32 * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = make_uint4(0, 0, 0, 0);
        if (j0 + 32 * u < d / 8 && !drop) v[u] = in16[j0 + 32 * u];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + 32 * u < d / 8) out[j0 + 32 * u] = v[u];
    }
  } else {
    const long long b = r / rows_per_b;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(dst) + ((size_t)(b * 3) * rows_per_b + (r - b * rows_per_b)) * dp;
    const size_t plane = (size_t)rows_per_b * dp;
    // four values a lane, eight loads of a row in flight (N 573, K 123, d 3969:
    // 10 us a copy against 38 with one at a time)
    constexpr int U = 8;
    const bool vec = d % 4 == 0 && (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    for (int j0 = 4 * lane; j0 < dp; j0 += 128 * U) {
      float v[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + 128 * u;
        if (vec) {
          const float4 w = j < d && !drop ? *reinterpret_cast<const float4 *>(in + j) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[u][0] = w.x, v[u][1] = w.y, v[u][2] = w.z, v[u][3] = w.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = j + i < d && !drop ? in[j + i] : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + 128 * u;
        if (j >= dp) break;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          __nv_bfloat162 h[2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat16 t = __float2bfloat16_rn(v[u][i]);
            const float f = __bfloat162float(t);
            // an infinity (or an overflow of the rounding) leaves no remainder
            v[u][i] = fabsf(f) < INFINITY ? v[u][i] - f : 0.f;
            if (i & 1) h[i / 2].y = t;
            else h[i / 2].x = t;
          }
          *reinterpret_cast<uint2 *>(out + p * plane + j) = *reinterpret_cast<const uint2 *>(h);
        }
      }
    }
  }
}

// Defined in fk_scores.cu / fk_scores_bias.cu, fk_join.cu and fk_operand.cu.
int launch_scores(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt, int *err,
                  cudaStream_t s);
int launch_scores_bias(const CUtensorMap &tx, const CUtensorMap &tc, const FwdSpace &f, const StatArgs &a, int fmt,
                       int *err, cudaStream_t s);
int launch_join(const JoinArgs &j, int dtype, cudaStream_t s);
int operand(const void *src, int dtype, long long rows, long long rows_per_b, int d, int dp, const float *bias,
            void *dst, cudaStream_t s);

}  // namespace soft
}  // namespace fk
