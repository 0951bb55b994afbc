// Joins the partial results of the score kernels, row by row.
//
// These kernels are resident while the score kernel still writes its partial
// results (it triggers its dependents at its start): what it writes is read with
// ordinary loads after pdl_wait(), never through the read-only path.  x, c and
// bias are older than the score kernel, and finished.
#include "fk_logprob.cuh"

namespace fk {
namespace soft {
namespace {

__device__ __forceinline__ void join_stats(float &m, float &s, float &u, float m2, float s2, float u2) {
  const float mm = fmaxf(m, m2);
  const float ms = mm == kNegInf ? 0.f : mm;
  // an empty side has s = u = 0 and its (clamped) distance contributes nothing;
  // a NaN sum stays NaN
  const float d1 = fmaxf(m - ms, kLowest), d2 = fmaxf(m2 - ms, kLowest);
  const float f1 = pow2(m - ms), f2 = pow2(m2 - ms);  // the m are whole numbers
  u = f1 * fmaf(d1, s, u) + f2 * fmaf(d2, s2, u2);
  s = f1 * s + f2 * s2;
  m = mm;
}

// Rounding must not make a log probability positive or an entropy negative.
// (NaN stays.)
__device__ __forceinline__ float at_least_0(float v) { return v < 0.f ? 0.f : v; }

// Scores of C columns in fp64, by LPR lanes, from the operands as given:
// products of 16-bit values are exact, and fp64 sums keep neighbours in rank
// apart that the fp32 accumulation cannot.
template <typename T, int LPR, int C>
__device__ __forceinline__ void exact_scores(const T *x, const T *c, const float *bias, float scale, const int (&k)[C],
                                             int d, bool vec, int lane, double (&s)[C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) s[i] = 0.0;
  constexpr int V = 16 / sizeof(T);
  if (vec) {
#pragma unroll(C <= 2 ? 4 : 2)
    for (int j = lane; j < d / V; j += LPR) {
      T xv[V], cv[C][V];
      *reinterpret_cast<uint4 *>(xv) = __ldg(reinterpret_cast<const uint4 *>(x) + j);
#pragma unroll
      for (int i = 0; i < C; ++i)
        *reinterpret_cast<uint4 *>(cv[i]) = __ldg(reinterpret_cast<const uint4 *>(c + (size_t)k[i] * d) + j);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const double xd = (double)to_f(xv[q]);
#pragma unroll
        for (int i = 0; i < C; ++i) s[i] = fma(xd, (double)to_f(cv[i][q]), s[i]);
      }
    }
  } else {
    for (int j = lane; j < d; j += LPR) {
      const double xd = (double)to_f(x[j]);
#pragma unroll
      for (int i = 0; i < C; ++i) s[i] = fma(xd, (double)to_f(c[(size_t)k[i] * d + j]), s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    s[i] *= (double)scale;
    if (bias) s[i] = bias[k[i]] == kNegInf ? (double)kNegInf : s[i] + (double)bias[k[i]];
  }
}

// The largest squared norm of a batch's table rows (float bits; they order as
// integers).
template <typename T>
__global__ void __launch_bounds__(256) k_max_norm(const T *c, long long rows, long long K, int d, unsigned *out) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  float s = 0.f;
  for (int j = lane; j < d; j += 32) {
    const float v = to_f(c[(size_t)r * d + j]);
    s = fmaf(v, v, s);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && s > 0.f) atomicMax(out + r / K, __float_as_uint(s));
}

constexpr int kJoinWarps = 8;
constexpr int kNoCol = 0x7fffffff;

// The best `n` of the lanes' sorted lists of up to LL columns (k < 0: the end);
// lane j of the group keeps the j-th.  The lists move up as their heads go.
template <int LPR, int LL>
__device__ __forceinline__ void draw(int n, int lane, float (&lv)[LL], int (&lk)[LL], float &mv, int &mk) {
  mv = kNegInf;
  mk = -1;
  for (int j = 0; j < n; ++j) {
    float v = lk[0] >= 0 ? lv[0] : kNegInf;
    int k = lk[0] >= 0 ? lk[0] : kNoCol;
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
    const bool won = lk[0] == k;
#pragma unroll
    for (int i = 0; i < LL; ++i) {
      lv[i] = won && i + 1 < LL ? lv[i + 1 < LL ? i + 1 : i] : lv[i];
      lk[i] = won ? (i + 1 < LL ? lk[i + 1 < LL ? i + 1 : i] : -1) : lk[i];
    }
  }
}

// Puts (v, k) behind what is better in a list: larger, or equal in a lower
// column (k < 0, the end of a list, orders after every column).
template <int LL>
__device__ __forceinline__ void insert_ordered(float (&hv)[LL], int (&hk)[LL], float v, int k) {
#pragma unroll
  for (int i = LL - 1; i >= 0; --i) {
    const int h = i > 0 ? i - 1 : 0;
    const bool below = v > hv[i] || (v == hv[i] && (unsigned)k < (unsigned)hk[i]);
    const bool shift = i > 0 && (v > hv[h] || (v == hv[h] && (unsigned)k < (unsigned)hk[h]));
    hk[i] = below ? (shift ? hk[h] : k) : hk[i];
    hv[i] = below ? (shift ? hv[h] : v) : hv[i];
  }
}

// A row's joined statistics: lse = m + ls in base 2 with m whole and ls in [0, 1)
// (ls = log2 of the sum's significand), so that a confident row's log
// probability is a small difference of small numbers.  An m of 2^23 or more in
// magnitude cannot take in the sum's exponent: ls is then log2 of the whole sum.
struct RowStat {
  float m, ls, hs;  // hs = (sum e (t - m)) / sum
  float sig;        // 2^ls
  bool none;        // every column is masked: lse = -inf, entropy 0
  bool nan;
};

__device__ __forceinline__ RowStat row_stat(float m, float s, float u) {
  RowStat r;
  r.none = m == kNegInf && s == 0.f;
  r.nan = !(s == s);
  r.hs = u / s;
  if (s > 0.f && s < INFINITY && fabsf(m) < kCoarse) {
    const int e = ilogbf(s);
    r.m = m + (float)e;
    r.sig = scalbnf(s, -e);
    r.ls = log2f(r.sig);
    r.hs -= (float)e;
  } else {
    r.m = m;
    r.sig = s;
    r.ls = log2f(s);
  }
  return r;
}

// Log probability of a stored score (a product, or in base 2 with a bias).  Of
// a column that holds more than half of the sum it is -log1p(what the others
// add / e): the sum has the same ex2.approx of the same score in it, whose error
// (2^-22 of it) cancels in the difference instead of standing beside a small result.
__device__ __forceinline__ float stored_logp(const JoinArgs &a, const RowStat &q, float v) {
  if (q.none || (v == kNegInf && !q.nan)) return kNegInf;
  const float rel = fabsf(q.m) >= kCoarse ? __fmul_rn(v, a.unit2) - q.m : fmaf(v, a.unit2, -q.m);
  const float e = ex2(rel);
  if (e + e > q.sig && q.sig < INFINITY) return -log1pf(fmaxf(q.sig - e, 0.f) / e);
  return -at_least_0((q.ls - rel) * kLn2);
}

__device__ __forceinline__ void write_stats(const JoinArgs &a, long long r, const RowStat &q, float tgt) {
  const int id = a.ids[r];
  const bool valid = id >= 0 && id < a.K;
  if (id >= a.K) atomicCAS(a.err, DEV_OK, DEV_BAD_ID);
  const double lse = q.none ? (double)kNegInf : ((double)q.m + (double)q.ls) * M_LN2;
  a.lse[r] = (float)lse;
  if (a.lse_rest) {
    const float rest = (float)(lse - (double)(float)lse);
    a.lse_rest[r] = rest == rest ? rest : 0.f;
  }
  if (a.entropy) a.entropy[r] = q.none ? 0.f : at_least_0((q.ls - q.hs) * kLn2);
  a.logp[r] = valid ? stored_logp(a, q, tgt) : 0.f;
}

__device__ __forceinline__ void write_top(const JoinArgs &a, long long r, int rank, int k, float v, const RowStat &q) {
  a.top_ids[r * a.top + rank] = k;
  a.top_logp[r * a.top + rank] = stored_logp(a, q, v);
}

// Twice what a stored score v of a row of squared norm n2 can be off: the
// roundings of its accumulation, (d / 16 + 16) 2^-23 |x| |c| (six times the
// steps for fp32 operands), and a few of its own.  Neighbours in rank further
// apart are settled; only closer ones are worth the loads of exact scores.
template <typename T>
__device__ __forceinline__ float rank_error(const JoinArgs &a, long long b, float n2, bool bias, float v) {
  const float unit = bias ? a.scale * kLog2e : 1.f;  // of the stored scores
  const float steps = (a.d / 16.f + 18.f) * (sizeof(T) == 4 ? 6.f : 1.f);
  const float size = unit * sqrtf(n2) * sqrtf(__uint_as_float(a.max_norm2[b]));
  return 2.f * ((steps + 4.f) * 1.2e-7f * size + 1e-6f * fabsf(v)) + 1e-37f;
}

// Joins the statistics of LPR lanes; all of them hold the result.
template <int LPR>
__device__ __forceinline__ void reduce_stats(float &m, float &s, float &u, float &tgt, int lane) {
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
}

// LPR lanes per row.
template <typename T, int LPR, int LL>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join(const JoinArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & (LPR - 1);
  const long long r0 = (long long)blockIdx.x * (kJoinWarps * (32 / LPR)) + threadIdx.x / LPR;
  // lanes of a row beyond the last one follow along on the last row
  const bool live = r0 < a.rows;
  const long long r = live ? r0 : a.rows - 1;
  const long long b = r / a.N;
  float m = kNegInf, s = 0.f, u = 0.f, tgt = kNegInf;
  for (int p = lane; p < a.parts; p += LPR) {
    const float4 q = a.part[r * a.parts + p];
    join_stats(m, s, u, q.x, q.y, q.z);
    tgt = fmaxf(tgt, q.w);
  }
  reduce_stats<LPR>(m, s, u, tgt, lane);
  const RowStat st = row_stat(m, s, u);
  if (live && lane == 0) write_stats(a, r, st, tgt);
  if (a.top == 0) return;

  // the lane's own list: its parts' lists, joined (LL columns at most)
  float hv[LL], mv;
  int hk[LL], mine;
#pragma unroll
  for (int i = 0; i < LL; ++i) {
    hv[i] = kNegInf;
    hk[i] = -1;
  }
  for (int p = lane; p < a.parts; p += LPR) {
    const float *pv = a.top_v + (r * a.parts + p) * a.L;
    const int32_t *pk = a.top_i + (r * a.parts + p) * a.L;
#pragma unroll 1
    for (int j = 0; j < LL; ++j) {
      const int k = pk[j];
      if (k < 0) break;
      insert_ordered<LL>(hv, hk, pv[j], k);
    }
  }
  __syncwarp();
  draw<LPR, LL>(a.cands, lane, hv, hk, mv, mine);
  const unsigned group = LPR == 32 ? 0u : (threadIdx.x & 31) & ~(LPR - 1u);  // first lane of the row's group
  const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << group;
  {
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
  const T *x = static_cast<const T *>(a.x) + (size_t)r * a.d;
  const T *c = static_cast<const T *>(a.c) + (size_t)b * a.K * a.d;
  const float *bias = a.bias ? a.bias + b * a.K : nullptr;
  if (a.max_norm2) {
    // many rows: see rank_error
    float n2 = 0.f;
    if (a.vec) {
      constexpr int V = 16 / sizeof(T);
      for (int j = lane; j < a.d / V; j += LPR) {
        T xv[V];
        *reinterpret_cast<uint4 *>(xv) = __ldg(reinterpret_cast<const uint4 *>(x) + j);
#pragma unroll
        for (int q = 0; q < V; ++q) n2 = fmaf(to_f(xv[q]), to_f(xv[q]), n2);
      }
    } else {
      for (int j = lane; j < a.d; j += LPR) n2 = fmaf(to_f(x[j]), to_f(x[j]), n2);
    }
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
    const float off = rank_error<T>(a, b, n2, bias != nullptr, mv);
    const float next = __shfl_down_sync(0xffffffffu, mv, 1, LPR);
    const bool close = lane < a.cands && (mv == kNegInf || (lane < a.top && lane + 1 < a.cands && !(mv - next > off)));
    if (!__any_sync(0xffffffffu, close)) {
      if (live && lane < a.top) {
        write_top(a, r, lane, mine, mv, st);
      }
      return;
    }
  }
  double v = (double)kNegInf;
  for (int j = 0; j < a.cands; j += 4) {
      int k[4];
      double e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = __shfl_sync(0xffffffffu, mine, min(j + i, a.cands - 1), LPR);
      exact_scores<T, LPR, 4>(x, c, bias, a.scale, k, a.d, a.vec, lane, e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane == j + i) v = e[i];
  }
  const double rank_v = v == v ? v : (double)kNegInf;
  int rank = 0;
  for (int j = 0; j < a.cands; ++j) {
    const double v2 = __shfl_sync(0xffffffffu, rank_v, j, LPR);
    const int k2 = __shfl_sync(0xffffffffu, mine, j, LPR);
    rank += v2 > rank_v || (v2 == rank_v && k2 < mine);
  }
  if (live && lane < a.cands && rank < a.top) {
    write_top(a, r, rank, mine, mv, st);
  }
}


// A block per row, for few rows: their lists are too many for a warp, and their
// exact scores would be one warp's long chain of loads.  The code is kept small
// rather than unrolled: one row runs it once, out of a cold instruction cache.
//
// Columns are ordered by a 64-bit key (score, then lowest index).  Every thread
// has the best of its lists; the cands-th best of these is a bound, and only
// columns at or above it are gathered (cands threads' lists at most) and ranked.
constexpr int kMaxParts = 3 * 2 * 160;  // of one row: three per run
constexpr int kGather = 32 * 32 * ((kMaxParts + 255) / 256);

__device__ __forceinline__ unsigned long long column_key(float v, int k) {
  if (k < 0) return 0ull;
  const unsigned b = __float_as_uint(v == 0.f ? 0.f : v);
  const unsigned o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return ((unsigned long long)o << 32) | (0xffffffffu - (unsigned)k);
}

__device__ __forceinline__ float key_score(unsigned long long key) {
  const unsigned o = (unsigned)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join_block(const JoinArgs a) {
  __shared__ float parts[4][kJoinWarps], stored[32];
  __shared__ unsigned long long heads[kJoinWarps * 32], bound, found[kGather];
  __shared__ int n_found, cand[32];
  __shared__ double exact[32];
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long r = blockIdx.x, b = r / a.N;
  if (tid == 0) {
    n_found = 0;
    bound = 0ull;
  }
  float m = kNegInf, s = 0.f, u = 0.f, tgt = kNegInf;
  unsigned long long head = 0ull;
  for (int p = tid; p < a.parts; p += 32 * kJoinWarps) {
    const float4 q = a.part[r * a.parts + p];
    const long long o = (r * a.parts + p) * a.L;
    head = max(head, column_key(a.top_v[o], a.top_i[o]));
    join_stats(m, s, u, q.x, q.y, q.z);
    tgt = fmaxf(tgt, q.w);
  }
  reduce_stats<32>(m, s, u, tgt, lane);
  if (lane == 0) parts[0][warp] = m, parts[1][warp] = s, parts[2][warp] = u, parts[3][warp] = tgt;
  // the warp's best heads, in order
  unsigned long long left = head;
#pragma unroll 1
  for (int j = 0; j < a.cands; ++j) {
    const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(left >> 32));
    const unsigned lo = __reduce_max_sync(0xffffffffu, (unsigned)(left >> 32) == hi ? (unsigned)left : 0u);
    const unsigned long long best = ((unsigned long long)hi << 32) | lo;
    if (lane == 0) heads[warp * a.cands + j] = best;
    if (left == best) left = 0ull;
  }
  __syncthreads();
  m = parts[0][0], s = parts[1][0], u = parts[2][0], tgt = parts[3][0];
#pragma unroll 1
  for (int w = 1; w < kJoinWarps; ++w) {
    join_stats(m, s, u, parts[0][w], parts[1][w], parts[2][w]);
    tgt = fmaxf(tgt, parts[3][w]);
  }
  const RowStat st = row_stat(m, s, u);
  if (tid == 0) write_stats(a, r, st, tgt);
  if (tid < kJoinWarps * a.cands) {
    const unsigned long long mine = heads[tid];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < kJoinWarps * a.cands; ++i) rank += heads[i] > mine;
    if (rank == a.cands - 1 && mine) bound = mine;  // keys differ: one thread at most
  }
  __syncthreads();
  const unsigned long long least = bound;
  if (head && head >= least) {
#pragma unroll 1
    for (int p = tid; p < a.parts; p += 32 * kJoinWarps) {
      const long long o = (r * a.parts + p) * a.L;
#pragma unroll 1
      for (int j = 0; j < a.L; ++j) {  // sorted: the rest is lower
        const unsigned long long key = column_key(a.top_v[o + j], a.top_i[o + j]);
        if (!key || key < least) break;
        found[atomicAdd(&n_found, 1)] = key;
      }
    }
  }
  __syncthreads();
  const int n = n_found;
#pragma unroll 1
  for (int i = tid; i < n; i += 32 * kJoinWarps) {
    const unsigned long long mine = found[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += found[j] > mine;
    if (rank < a.cands) {
      cand[rank] = (int)(0xffffffffu - (unsigned)mine);
      stored[rank] = key_score(mine);
    }
  }
  __syncthreads();
  if (n < a.cands) {  // masked (or NaN) columns are in no list: they follow, lowest index first
    if (tid == 0) {
      int next = 0;
      for (int i = n; i < a.cands; ++i, ++next) {
        for (int j = 0; j < n; ++j)
          if (cand[j] == next) {
            ++next;
            j = -1;
          }
        cand[i] = next;
        stored[i] = kNegInf;
      }
    }
    __syncthreads();
  }
  const T *x = static_cast<const T *>(a.x) + (size_t)r * a.d;
  const T *c = static_cast<const T *>(a.c) + (size_t)b * a.K * a.d;
  const float *bias = a.bias ? a.bias + b * a.K : nullptr;
#pragma unroll 1
  for (int j = warp; j < a.cands; j += 2 * kJoinWarps) {  // candidates j and j + 8
    const int other = j + kJoinWarps < a.cands ? j + kJoinWarps : j;
    const int k[2] = {cand[j], cand[other]};
    double e[2];
    if (other == j) {
      const int k1[1] = {k[0]};
      double e1[1];
      exact_scores<T, 32, 1>(x, c, bias, a.scale, k1, a.d, a.vec, lane, e1);
      e[0] = e1[0];
    } else {
      exact_scores<T, 32, 2>(x, c, bias, a.scale, k, a.d, a.vec, lane, e);
    }
    if (lane == 0) {
      exact[j] = e[0];
      if (other != j) exact[other] = e[1];
    }
  }
  __syncthreads();
  if (tid < a.cands) {
    const double v = exact[tid], rank_v = v == v ? v : (double)kNegInf;
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j < a.cands; ++j) {
      const double w = exact[j], wv = w == w ? w : (double)kNegInf;
      rank += wv > rank_v || (wv == rank_v && cand[j] < cand[tid]);
    }
    if (rank < a.top) write_top(a, r, rank, cand[tid], stored[tid], st);
  }
}

// Many rows of few parts: a thread per row.  LL = 0: statistics only.  Three CTAs an
// SM with the shortest lists: three registers more cost the third, and 604800 rows 2%.
template <typename T, int LL>
__global__ void __launch_bounds__(256, LL <= 4 ? 3 : 1) k_join_rows(const JoinArgs a) {
  pdl_wait();
  constexpr int C = LL ? LL : 1;
  const int lane = threadIdx.x & 31;
  const long long r0 = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool live = r0 < a.rows;
  const long long r = live ? r0 : a.rows - 1, b = r / a.N;
  float m = kNegInf, s = 0.f, u = 0.f, tgt = kNegInf;
  for (int p = 0; p < a.parts; ++p) {
    const float4 q = a.part[r * a.parts + p];
    join_stats(m, s, u, q.x, q.y, q.z);
    tgt = fmaxf(tgt, q.w);
  }
  const RowStat st = row_stat(m, s, u);
  if (live) write_stats(a, r, st, tgt);
  if (LL == 0) return;

  float hv[C];
  int hk[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    hv[i] = kNegInf;
    hk[i] = -1;
  }
  for (int p = 0; p < a.parts; ++p) {
    const float4 *pv = reinterpret_cast<const float4 *>(a.top_v + (r * a.parts + p) * a.L);
    const int4 *pk = reinterpret_cast<const int4 *>(a.top_i + (r * a.parts + p) * a.L);
#pragma unroll
    for (int q = 0; q < C / 4; ++q) {
      const float4 v4 = pv[q];
      const int4 k4 = pk[q];
      const float nv[4] = {v4.x, v4.y, v4.z, v4.w};
      const int nk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // lists are sorted: once nobody's next column enters, the rest do not either
        const bool in = nv[j] > hv[C - 1] || (nv[j] == hv[C - 1] && (unsigned)nk[j] < (unsigned)hk[C - 1]);
        if (__any_sync(0xffffffffu, in)) insert_ordered<C>(hv, hk, nv[j], nk[j]);
      }
    }
  }
  const T *x = static_cast<const T *>(a.x) + (size_t)r * a.d;
  const float *bias = a.bias ? a.bias + b * a.K : nullptr;
  float n2 = 0.f;
  if (a.vec) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll 4
    for (int j = 0; j < a.d / V; ++j) {
      T xv[V];
      *reinterpret_cast<uint4 *>(xv) = __ldg(reinterpret_cast<const uint4 *>(x) + j);
#pragma unroll
      for (int q = 0; q < V; ++q) n2 = fmaf(to_f(xv[q]), to_f(xv[q]), n2);
    }
  } else {
    for (int j = 0; j < a.d; ++j) n2 = fmaf(to_f(x[j]), to_f(x[j]), n2);
  }
  bool close = false;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (i < a.cands) close |= hk[i] < 0;
    if (i + 1 < C && i < a.top && i + 1 < a.cands)
      close |= !(hv[i] - hv[i + 1 < C ? i + 1 : i] > rank_error<T>(a, b, n2, bias != nullptr, hv[i]));
  }
  if (live && !close) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < a.top) write_top(a, r, i, hk[i], hv[i], st);
  }
  // rows whose order is open, one after another by the whole warp
  for (unsigned open = __ballot_sync(0xffffffffu, live && close); open; open &= open - 1) {
    const int src = __ffs(open) - 1;
    const long long rs = __shfl_sync(0xffffffffu, r, src), bs = rs / a.N;
    const T *xs = static_cast<const T *>(a.x) + (size_t)rs * a.d;
    const T *cs = static_cast<const T *>(a.c) + (size_t)bs * a.K * a.d;
    const float *bb = a.bias ? a.bias + bs * a.K : nullptr;
    if (lane == src) {  // masked (or NaN) columns are in no list: they follow, lowest index first
      int next = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (i < a.cands && hk[i] < 0) {
          for (bool used = true; used;) {
            used = false;
#pragma unroll
            for (int j = 0; j < C; ++j) used |= hk[j] == next;
            next += used;
          }
          hk[i] = next++;
        }
      }
    }
    double ev[C];
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      int k[4];
      double e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = max(__shfl_sync(0xffffffffu, hk[i + j < C ? i + j : 0], src), 0);
      exact_scores<T, 32, 4>(xs, cs, bb, a.scale, k, a.d, a.vec, lane, e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < C) ev[i + j < C ? i + j : 0] = e[j];
    }
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const double vi = ev[i] == ev[i] ? ev[i] : (double)kNegInf;
        int rank = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const double vj = ev[j] == ev[j] ? ev[j] : (double)kNegInf;
          rank += j < a.cands && (vj > vi || (vj == vi && hk[j] < hk[i]));
        }
        if (i < a.cands && rank < a.top) write_top(a, r, rank, hk[i], hv[i], st);
      }
    }
  }
}

template <typename T, int LPR, int LL>
int launch_join_as(const JoinArgs &j, cudaStream_t s) {
  FK_CUDA(launch_pdl(k_join<T, LPR, LL>, dim3((unsigned)cdiv(j.rows, kJoinWarps * (32 / LPR))), dim3(32 * kJoinWarps), 0,
                     s, j));
  return launched();
}

// Many rows: a thread per row where its parts are few (604800 rows of 3 parts,
// top 4: 185 us against 246 by 8 lanes a row); else as many lanes as there are
// candidates, at least 8.
template <typename T, int LL>
int launch_join_many(const JoinArgs &j, cudaStream_t s) {
  if (j.max_norm2) {
    FK_CUDA(cudaMemsetAsync(j.max_norm2, 0, (size_t)(j.rows / j.N) * sizeof(unsigned), s));
    const long long rows = j.rows / j.N * j.K;
    FK_CUDA(launch_pdl(k_max_norm<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const T *>(j.c), rows,
                       j.K, j.d, j.max_norm2));
    FK_TRY(launched());
  }
  if constexpr (LL <= 16) {
    if (j.rows > kJoinBlockRows && j.parts <= 8) {
      const dim3 grid((unsigned)cdiv(j.rows, 256));
      if (j.L) FK_CUDA(launch_pdl(k_join_rows<T, LL>, grid, dim3(256), 0, s, j));
      else FK_CUDA(launch_pdl(k_join_rows<T, 0>, grid, dim3(256), 0, s, j));
      return launched();
    }
  }
  if (j.cands <= 8 && j.parts <= 64) return launch_join_as<T, 8, LL>(j, s);
  if (j.cands <= 16 && j.parts <= 64) return launch_join_as<T, 16, LL>(j, s);
  return launch_join_as<T, 32, LL>(j, s);
}

// A block per row while the rows alone do not fill the SMs.
template <typename T>
int launch_join_typed(const JoinArgs &j, cudaStream_t s) {
  if (j.L && j.rows <= kJoinBlockRows) {
    if (j.parts > kMaxParts) return set_error(FK_EUNSUPPORTED, "too many partial results per row");
    FK_CUDA(launch_pdl(k_join_block<T>, dim3((unsigned)j.rows), dim3(32 * kJoinWarps), 0, s, j));
    return launched();
  }
  if (j.L <= 4) return launch_join_many<T, 4>(j, s);
  if (j.L == 8) return launch_join_many<T, 8>(j, s);
  if (j.L == 12) return launch_join_many<T, 12>(j, s);
  if (j.L == 16) return launch_join_many<T, 16>(j, s);
  return launch_join_many<T, 32>(j, s);
}

}  // namespace

int launch_join(const JoinArgs &j, int dtype, cudaStream_t s) {
  if (dtype == FK_F32) return launch_join_typed<float>(j, s);
  if (dtype == FK_BF16) return launch_join_typed<__nv_bfloat16>(j, s);
  return launch_join_typed<__half>(j, s);
}

}  // namespace soft
}  // namespace fk
