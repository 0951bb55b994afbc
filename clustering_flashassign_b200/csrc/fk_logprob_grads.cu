// Gradients of the token log probabilities.
#include "fk_logprob.cuh"

namespace fk {
namespace soft {
namespace {

// ------------------------------------------------------------------ backward
// Coefficients of every row (a warp each), its copy for the products (see
// fk_operand.cu: a row without any gradient becomes zero), and the largest
// bound of |G| over the rows (float bits; positive floats order as integers).
template <typename T>
__global__ void __launch_bounds__(256)
    k_rows(const int32_t *ids, const float *lse, const float *lse_rest, const float *entropy, const float *dlogp, const float *dlse,
           const float *dent, long long rows, long long rows_per_b, int K, RowGrad *out, unsigned *bound, const T *x,
           int d, int dp, void *xs, int *err) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  RowGrad g = {};
  g.id = ids[r];
  if (g.id >= K && lane == 0) atomicCAS(err, DEV_OK, DEV_BAD_ID);
  if (g.id < 0 || g.id >= K) g.id = -1;
  g.a = dlogp && g.id >= 0 ? dlogp[r] : 0.f;
  float l = dlse ? dlse[r] : 0.f, e = dent ? dent[r] : 0.f;
  const float v = lse[r];
  if (v == kNegInf) g.a = l = e = 0.f;  // every column is masked
  if (g.a == 0.f && l == 0.f && e == 0.f) g.id = -2;
  const double lse2 = ((double)v + (lse_rest ? (double)lse_rest[r] : 0.0)) * 1.4426950408889634;
  g.lse2 = (float)lse2;
  // lse and lse_rest hold 2^-47 of the logarithm.  Beyond 2^31, scores are 256
  // apart or equal: the row is even over its largest ones, g.lse2 is their score
  // and the logarithm of their number is the entropy.
  float lo = v == kNegInf ? 0.f : (float)(lse2 - (double)g.lse2);
  if (fabs(lse2) >= 2147483648.0) lo = entropy ? entropy[r] * kLog2e : fabs(lse2) < 140737488355328.0 ? lo : 0.f;
  const float f = exp2f(-lo);
  g.c1 = f * (l - g.a - e * (dent ? entropy[r] : 0.f) + e * kLn2 * lo);
  g.c2 = -f * e * kLn2;
  if (lane == 0) {
    out[r] = g;
    // |p (log p + H)| <= max(1 / e, log K) <= log K + 1
    const float big = fabsf(g.a) + fabsf(l) + fabsf(e) * (logf((float)K) + 1.f);
    // a row whose gradient overflowed does not take the others' scale
    if (bound && big > 0.f && big < INFINITY) atomicMax(bound, __float_as_uint(big));
  }
  copy_row<T>(x, r, rows_per_b, d, dp, g.id == -2, xs, lane);
}

// The power of two that brings `bound` to [2^13, 2^14), within [2^-100, 2^100].
__device__ __forceinline__ float grad_scale(unsigned bound) {
  const float b = __uint_as_float(bound);
  if (!(b > 0.f)) return 1.f;
  int e = 13 - ilogbf(b);
  e = e < -100 ? -100 : e > 100 ? 100 : e;
  return ldexpf(1.f, e);
}

// A warp's 32 x 32 values (a row per thread) to 32 rows of memory, through
// shared memory, so that an instruction writes 64 (16-bit) or 128 bytes of each
// of its rows instead of 16: a third of the write transactions (N 16, K 131072,
// d 4096: dC 375 us against 718).  Rows in shared memory are 16 bytes apart from
// a multiple of 128, which spreads them over the banks.
template <typename T>
struct RowStore {
  static constexpr int kPitch = 32 * sizeof(T) + 16;
  static constexpr int kBytes = 32 * kPitch;  // per warp
  static constexpr int kPer = 16 / sizeof(T);  // values of one access
  static constexpr int kSegs = 32 / kPer;      // accesses of one row
  uint8_t *buf;

  __device__ __forceinline__ void put(const T (&v)[32], int lane) {
    uint4 *dst = reinterpret_cast<uint4 *>(buf + lane * kPitch);
#pragma unroll
    for (int i = 0; i < kSegs; ++i) dst[i] = reinterpret_cast<const uint4 *>(v)[i];
    __syncwarp();
  }
  // f(row of the 32, first of kPer columns, its values)
  template <class F>
  __device__ __forceinline__ void each(int lane, F f) {
#pragma unroll
    for (int i = 0; i < kSegs; ++i) {
      const int row = i * (32 / kSegs) + lane / kSegs, seg = lane % kSegs;
      T v[kPer];
      *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(buf + row * kPitch + seg * 16);
      f(row, seg * kPer, v);
    }
    __syncwarp();
  }
};

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
  static constexpr int kSeg = SEG ? tile::kSegBlocks : 0;
  static constexpr int kRegs = 152;
  const Args &a;
  const int r, lane;
  BiasTile bt;
  RowStore<T> rs;
  const float *bias = nullptr;
  RowGrad q = {};
  long long row = 0, top = 0;  // the thread's row, the warp's first
  float gs = 1.f;
  T *g = nullptr;
  float *cp = nullptr;

  __device__ GradEpi(const Args &args, int lane_, int r_in_tile, int third, uint8_t *smem)
      : a(args), r(r_in_tile), lane(lane_) {
    const int warp = third * 4 + r_in_tile / 32;
    rs.buf = smem + warp * RowStore<T>::kBytes;
    bt.sb = reinterpret_cast<float *>(smem + tile::kEpiWarps * RowStore<T>::kBytes) + warp * BiasTile::kFloats;
    if (args.bound) gs = grad_scale(*args.bound);
  }
  __device__ void begin(const Unit &w, long long row0) {
    row = row0 + r;
    q = RowGrad{};
    q.id = -2;
    if (row < a.nr) q = a.rows[w.b * a.row_stride + row];
    if (BIAS) bias = a.bias + w.b * a.K;
    top = row0 + (r & ~31);
    g = static_cast<T *>(a.g) + ((size_t)w.b * a.planes * a.nr + top) * a.Kp;
    const long long blk = (row0 + (r & ~31)) >> 5;
    cp = a.colpart && blk < a.nblk ? a.colpart + (w.b * a.nblk + blk) * a.Kp : nullptr;
  }
  static size_t smem_bytes() {
    return tile::kEpiWarps * (RowStore<T>::kBytes + (BIAS ? BiasTile::kFloats * 4 : 0));
  }
  __device__ __forceinline__ void prepare(long long col0, int stride) {
    if (BIAS) bt.load(bias, col0, stride, a.K, lane);
  }
  __device__ __forceinline__ bool skip(long long col) const { return col >= a.Kp; }
  __device__ __forceinline__ void chunk(const float (&acc)[32], long long col, int i) {
    {
      float v[32];
      const bool some_masked = scores32<BIAS>(acc, a.scale2, bt, i, col, a.K, v);
      const bool coarse = !BIAS && fabsf(q.lse2) >= kCoarse;
      if (!BIAS && __any_sync(0xffffffffu, coarse)) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = coarse ? __fmul_rn(v[j], a.scale2) : v[j];
      }
      const float s1 = coarse ? 1.f : a.scale2;
      const float2 nl = make_float2(-q.lse2, -q.lse2), sc = make_float2(s1, s1);
      const float2 c1 = make_float2(q.c1, q.c1), c2 = make_float2(q.c2, q.c2);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 w = make_float2(v[2 * j], v[2 * j + 1]);
        float2 lp2 = BIAS ? __fadd2_rn(w, nl) : __ffma2_rn(w, sc, nl);
        const float2 p = make_float2(ex2(lp2.x), ex2(lp2.y));
        if (some_masked) lp2 = make_float2(fmaxf(lp2.x, kLowest), fmaxf(lp2.y, kLowest));
        const float2 y = __fmul2_rn(p, __ffma2_rn(lp2, c2, c1));
        v[2 * j] = y.x;
        v[2 * j + 1] = y.y;
      }
      if (__any_sync(0xffffffffu, q.id == -2)) {  // rows without any gradient among the 32
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (q.id == -2) v[j] = 0.f;
      }
      const unsigned rel = (unsigned)(q.id - (int)col);
      if (__any_sync(0xffffffffu, rel < 32u)) {  // the target's own term, unless it is masked
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (rel == (unsigned)j && !(BIAS && bt.sb[i * 32 + j] == kNegInf)) v[j] += q.a;
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
      if (gs != 1.f) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= gs;
      }
#pragma unroll 1
      for (int pl = 0; pl < a.planes; ++pl) {
        T h[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          h[j] = from_f<T>(v[j]);
          v[j] -= to_f(h[j]);  // the next plane's value
        }
        rs.put(h, lane);
        T *dst = g + (size_t)pl * a.nr * a.Kp + col;
        rs.each(lane, [&](int row, int at, const T (&w)[RowStore<T>::kPer]) {
          if (top + row < a.nr && col + at < a.Kp)
            *reinterpret_cast<uint4 *>(dst + row * a.Kp + at) = *reinterpret_cast<const uint4 *>(w);
        });
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

template <typename T, int SEG>
struct StoreEpi {
  using Args = StoreArgs;
  static constexpr int kSeg = SEG;
  static constexpr int kRegs = 152;
  const Args &a;
  const int r, lane;
  float alpha;
  long long top = 0;  // the warp's first row
  T *out = nullptr;
  float *part = nullptr;
  uint8_t *buf;
  bool vec_t, vec_f;

  __device__ StoreEpi(const Args &args, int lane_, int r_in_tile, int third, uint8_t *smem)
      : a(args), r(r_in_tile), lane(lane_) {
    alpha = args.alpha;
    if (args.bound) alpha /= grad_scale(*args.bound);
    buf = smem + (third * 4 + r_in_tile / 32) * (args.part ? RowStore<float>::kBytes : RowStore<T>::kBytes);
    vec_t = (args.pitch * sizeof(T)) % 16 == 0;
    vec_f = args.cols % 4 == 0;
  }
  static size_t smem_bytes(bool parts) {
    return tile::kEpiWarps * (parts ? RowStore<float>::kBytes : RowStore<T>::kBytes);
  }
  __device__ void begin(const Unit &w, long long row0) {
    top = row0 + (r & ~31);
    out = static_cast<T *>(a.out) + w.b * a.batch_stride + top * a.pitch;
    if (a.part) part = a.part + w.ks * a.slot + (w.b * a.rows + top) * a.cols;
  }
  __device__ __forceinline__ void prepare(long long, int) {}
  __device__ __forceinline__ bool skip(long long col) const { return col >= a.cols; }

  template <typename S>
  __device__ __forceinline__ void store(const float (&acc)[32], long long col, S *base, long long pitch, bool vec,
                                        bool add) {
    RowStore<S> rs{buf};
    S h[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) h[j] = from_f<S>(acc[j] * alpha);
    rs.put(h, lane);
    rs.each(lane, [&](int row, int at, S (&w)[RowStore<S>::kPer]) {
      const long long left = a.cols - col - at;
      if (top + row >= a.rows || left <= 0) return;
      S *dst = base + row * pitch + col + at;
      if (vec && left >= RowStore<S>::kPer) {
        if (sizeof(S) == 4 && add) {
          S old[RowStore<S>::kPer];
          *reinterpret_cast<uint4 *>(old) = *reinterpret_cast<const uint4 *>(dst);
#pragma unroll
          for (int j = 0; j < RowStore<S>::kPer; ++j) w[j] = from_f<S>(to_f(w[j]) + to_f(old[j]));
        }
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(w);
      } else {
#pragma unroll
        for (int j = 0; j < RowStore<S>::kPer; ++j)
          if (j < left) dst[j] = sizeof(S) == 4 && add ? from_f<S>(to_f(w[j]) + to_f(dst[j])) : w[j];
      }
    });
  }
  __device__ __forceinline__ void chunk(const float (&acc)[32], long long col, int) {
    if (a.part) store<float>(acc, col, part, a.cols, vec_f, a.add);
    else store<T>(acc, col, out, a.pitch, vec_t, false);
  }
  __device__ void end(const Unit &) {}
};

// out = the sum of the parts, in order; four columns a thread where rows allow it.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    k_sum_parts(const float *part, int parts, long long slot, long long n, T *out) {
  pdl_wait();
  const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (i >= n) return;
  float s[V] = {};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    float v[V];
    if constexpr (V == 4) *reinterpret_cast<float4 *>(v) = __ldcs(reinterpret_cast<const float4 *>(part + p * slot + i));
    else v[0] = part[p * slot + i];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] += v[j];
  }
  T h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) h[j] = from_f<T>(s[j]);
  if constexpr (V == 4 && sizeof(T) == 2) *reinterpret_cast<uint2 *>(out + i) = *reinterpret_cast<uint2 *>(h);
  else if constexpr (V == 4) *reinterpret_cast<float4 *>(out + i) = *reinterpret_cast<float4 *>(h);
  else out[i] = h[0];
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
  const long long row_bytes = m.Kp * 2 * m.g_planes;
  f.nr = std::min<long long>(std::max<long long>(m.N, 1), std::max<long long>(256, kGradBudget / row_bytes / 256 * 256));
  f.bn = f.nr < m.N ? 1 : (int)std::max<long long>(1, std::min<long long>(m.B, kGradBudget / (row_bytes * f.nr)));
  f.pg = plan_runs(f.bn, f.nr, m.Kp, m.d, m.pairs, m.planes, m.dp * 2 * m.planes);
  f.px = plan_splits(f.bn, f.nr, m.d, m.K, m.g_pairs, m.g_planes, m.planes);
  f.pw = plan_splits(f.bn, m.K, m.d, f.nr, m.g_pairs, m.g_planes, m.planes);
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

// Partial sums of (B, rows, d) values, contiguous like the result.
template <typename T>
int launch_sum_parts(const float *part, int parts, long long n, int d, void *out, cudaStream_t s) {
  T *o = static_cast<T *>(out);
  if (d % 4 == 0 && n >= 1 << 20) {  // fewer values: one a thread keeps more loads in flight
    FK_CUDA(launch_pdl(k_sum_parts<T, 4>, dim3((unsigned)cdiv(n, 1024)), dim3(256), 0, s, part, parts, n, n, o));
  } else {
    FK_CUDA(launch_pdl(k_sum_parts<T, 1>, dim3((unsigned)cdiv(n, 256)), dim3(256), 0, s, part, parts, n, n, o));
  }
  return launched();
}

// dX or dC: a product with G, in segments where it is long.
template <typename T, bool A_MN>
int launch_product(const CUtensorMap &ta, const CUtensorMap &tb, const Plan &p, const StoreArgs &a, int fmt, int *err,
                   cudaStream_t s) {
  constexpr int kSeg = sizeof(T) == 4 ? tile::kSegBlocks : tile::kLongSegBlocks;
  if constexpr (sizeof(T) == 2) {
    if (cdiv((long long)p.pairs * p.kblocks, p.ksplits) <= kSeg)
      return launch_tiles<StoreEpi<T, 0>, A_MN, true>(ta, tb, p, a, StoreEpi<T, 0>::smem_bytes(a.part), fmt, err, s);
  }
  return launch_tiles<StoreEpi<T, kSeg>, A_MN, true>(ta, tb, p, a, StoreEpi<T, kSeg>::smem_bytes(a.part), fmt, err, s);
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
      ga.planes = m.g_planes;
      ga.colpart = dbias ? f.colpart : nullptr;
      ga.nblk = cdiv(nr, 32);
      // the forward pass's scores, summed in the same segments: p is normalised by
      // their lse, and of a confident row's 1 - p a difference of 1e-4 would be all
      // that is seen (one chain of 2048 terms: 3e-6 of the score)
      if (pg.kblocks * pg.pairs > tile::kSegBlocks)
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
        FK_TRY(map_16(&tg, f.g, bf, m.Kp, nr, (long long)bn * m.g_planes, m.Kp, nr * m.Kp, tile::kK, tile::kRows));
        FK_TRY(map_16(&tcm, (const char *)cmul + coff, bf, m.dp, m.K, (long long)bn * m.planes, m.dp,
                      (long long)m.K * m.dp, 64, tile::kK));
        Plan px = f.px;
        if (bn != f.bn || nr != f.nr) {
          px = plan_splits(bn, nr, m.d, m.K, m.g_pairs, m.g_planes, m.planes);
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
        FK_TRY((launch_product<T, false>(tg, tcm, px, sa, fmt, err, s)));
        if (sa.part)
          FK_TRY(launch_sum_parts<T>(f.partx, px.ksplits, sa.slot, m.d, sa.out, s));
      }
      // dc = G^T X: the contraction is the rows
      if (dc) {
        CUtensorMap tg, txm;
        FK_TRY(map_16(&tg, f.g, bf, m.Kp, nr, (long long)bn * m.g_planes, m.Kp, nr * m.Kp, 64, tile::kK));
        FK_TRY(map_16(&txm, (const char *)f.xs + xoff, bf, m.dp, nr, (long long)bn * m.planes, m.dp, m.N * m.dp, 64,
                      tile::kK));
        Plan pw = f.pw;
        if (bn != f.bn || nr != f.nr) {
          // the partial sums keep their slots over all blocks of rows
          pw = plan_splits(bn, m.K, m.d, nr, m.g_pairs, m.g_planes, m.planes);
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
        FK_TRY((launch_product<T, true>(tg, txm, pw, sa, fmt, err, s)));
        if (sa.part && r0 + nr >= m.N) {
          FK_TRY(launch_sum_parts<T>(f.partw, f.nr < m.N ? f.pw.ksplits : pw.ksplits, sa.slot, m.d, sa.out, s));
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
}  // namespace soft
}  // namespace fk

using namespace fk;
using namespace fk::soft;

extern "C" {

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
                        const int32_t *ids, const float *lse, const float *lse_rest, const float *entropy,
                        const float *dlogp, const float *dlse, const float *dentropy, void *dx, void *dc, float *dbias, void *workspace,
                        long long workspace_bytes, fk_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FK_TRY(check_soft(shape, scale));
  if (dbias && !bias) return set_error(FK_EINVAL, "dbias without bias");
  long long need = 0;
  FK_TRY(fk_logprob_backward_workspace(shape, bias != nullptr, dbias != nullptr, &need));
  const Dims m = dims_of(*shape);
  const bool al = m.dtype != FK_F32;
  FK_TRY(check_ptr(c, "c", al));
  if (dc) FK_TRY(check_ptr(dc, "dc", true));
  if (m.N > 0) {
    FK_TRY(check_ptr(x, "x", al));
    FK_TRY(check_ptr(ids, "ids", false));
    FK_TRY(check_ptr(lse, "lse", false));
    if (dentropy) FK_TRY(check_ptr(entropy, "entropy", false));
    if (dx) FK_TRY(check_ptr(dx, "dx", true));
    FK_TRY(check_ptr(workspace, "workspace", true));
    if (workspace_bytes < need)
      return set_error(FK_EINVAL, "workspace is smaller than fk_logprob_backward_workspace asks for");
  }
  FK_TRY(check_dev_opt(dc, "dc"));
  FK_TRY(check_dev_opt(dbias, "dbias"));
  if (m.N == 0) {  // no rows: the table's gradients are zero
    if (dc) FK_CUDA(cudaMemsetAsync(dc, 0, (size_t)m.B * m.K * m.d * esize(m.dtype), s));
    if (dbias) FK_CUDA(cudaMemsetAsync(dbias, 0, (size_t)m.B * m.K * 4, s));
    return FK_OK;
  }
  FK_TRY(check_dev_opt(dx, "dx"));
  FK_TRY(check_dev(x, "x"));
  FK_TRY(check_dev(c, "c"));
  FK_TRY(check_dev_opt(bias, "bias"));
  FK_TRY(check_dev(ids, "ids"));
  FK_TRY(check_dev(lse, "lse"));
  FK_TRY(check_dev_opt(lse_rest, "lse_rest"));
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
  unsigned *bound = m.dtype == FK_F16 ? f.bound : nullptr;  // fp16 alone needs G scaled
  if (bound) FK_CUDA(cudaMemsetAsync(bound, 0, 16, s));
  auto prepare = [&](auto tag) -> int {
    using T = decltype(tag);
    FK_CUDA(launch_pdl(k_rows<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, ids, lse, lse_rest, entropy, dlogp,
                       dlse, dentropy, rows, m.N, m.K, f.rows, bound, static_cast<const T *>(x), m.d, m.dp, f.xs, err));
    return launched();
  };
  if (m.dtype == FK_F32) FK_TRY(prepare(float{}));
  else FK_TRY(prepare(__half{}));  // 16-bit rows are copied as bits
  if (f.cs) FK_TRY(operand(c, m.dtype, (long long)m.B * m.K, m.K, m.d, m.dp, bias, f.cs, s));
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
