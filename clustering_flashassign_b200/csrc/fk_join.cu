// Joins the partial results of the score kernels, row by row.
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
  const float f1 = ex2(m - ms), f2 = ex2(m2 - ms);
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
#pragma unroll(C == 1 ? 4 : 2)
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

// One warp's joined lists (and the row's candidates with their exact scores)
// where eight warps share a row.
struct JoinRow {
  float m[kJoinWarps], s[kJoinWarps], u[kJoinWarps], tgt[kJoinWarps];
  float v[kJoinWarps][32];
  int k[kJoinWarps][32];
  int cand[32];
  double exact[32];
};

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

__device__ __forceinline__ void write_stats(const JoinArgs &a, long long r, float m, float s, float u, float tgt,
                                            bool none, float ls) {
  const int id = a.ids[r];
  const bool valid = id >= 0 && id < a.K;
  if (id >= a.K) atomicCAS(a.err, DEV_OK, DEV_BAD_ID);
  a.lse[r] = none ? kNegInf : (m + ls) * kLn2;
  if (a.entropy) a.entropy[r] = none ? 0.f : at_least_0((ls - u / s) * kLn2);
  a.logp[r] = !valid ? 0.f : (none || (tgt == kNegInf && s == s)) ? kNegInf : -at_least_0((ls - (tgt - m)) * kLn2);
}

__device__ __forceinline__ void write_top(const JoinArgs &a, long long r, int rank, int k, double v, float m, float s,
                                          bool none, float ls) {
  const float lp = (float)(v - (double)(none ? kNegInf : m) * M_LN2) - ls * kLn2;
  a.top_ids[r * a.top + rank] = k;
  a.top_logp[r * a.top + rank] = v == (double)kNegInf && s == s ? kNegInf : -at_least_0(-lp);
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

// LPR lanes of WPR warps per row.  (8, 1): many rows of few parts, four rows a
// warp; (32, 1); (32, 8): few rows, whose exact scores would otherwise be one
// warp's long chain of loads.
template <typename T, int LPR, int WPR, int LL>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join(const JoinArgs a) {
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
    write_stats(a, r, m, s, u, tgt, none, ls);
  }
  if (a.top == 0) return;

  // the lane's own list: its parts' lists, joined (LL columns at most)
  float hv[LL], mv;
  int hk[LL], mine;
#pragma unroll
  for (int i = 0; i < LL; ++i) {
    hv[i] = kNegInf;
    hk[i] = -1;
  }
  for (int p = first; p < a.parts; p += step) {
    const float4 *pv = reinterpret_cast<const float4 *>(a.top_v + (r * a.parts + p) * a.L);
    const int4 *pk = reinterpret_cast<const int4 *>(a.top_i + (r * a.parts + p) * a.L);
    float nv[LL];
    int nk[LL];
#pragma unroll
    for (int i = 0; i < LL / 4; ++i) {
      const float4 v = __ldg(pv + i);
      const int4 k = __ldg(pk + i);
      nv[4 * i] = v.x, nv[4 * i + 1] = v.y, nv[4 * i + 2] = v.z, nv[4 * i + 3] = v.w;
      nk[4 * i] = k.x, nk[4 * i + 1] = k.y, nk[4 * i + 2] = k.z, nk[4 * i + 3] = k.w;
    }
    if (p == first) {
#pragma unroll
      for (int i = 0; i < LL; ++i) {
        hv[i] = nv[i];
        hk[i] = nk[i];
      }
    } else {
#pragma unroll(LL <= 16 ? LL : 1)
      for (int j = 0; j < LL; ++j) {
        insert_ordered<LL>(hv, hk, nv[j], nk[j]);
      }
    }
  }
  draw<LPR, LL>(a.cands, lane, hv, hk, mv, mine);
  if (WPR > 1) {
    sh.v[warp][lane] = mv;
    sh.k[warp][lane] = mine;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < LL; ++i) {
        hv[i] = lane < WPR ? sh.v[lane < WPR ? lane : 0][i] : kNegInf;
        hk[i] = lane < WPR ? sh.k[lane < WPR ? lane : 0][i] : -1;
      }
      draw<LPR, LL>(a.cands, lane, hv, hk, mv, mine);
    }
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
  if (WPR == 1 && a.max_norm2) {
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
        a.top_ids[r * a.top + lane] = mine;
        a.top_logp[r * a.top + lane] = -at_least_0((ls - (mv * (bias ? 1.f : a.scale * kLog2e) - m)) * kLn2);
      }
      return;
    }
  }
  double v = (double)kNegInf;
  if (WPR > 1) {  // candidates warp, warp + 8, ...
    if (warp < a.cands) {
      int k[4];
      double e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = sh.cand[warp + 8 * i < a.cands ? warp + 8 * i : warp];
      if (a.cands <= 8) {
        const int k1[1] = {k[0]};
        double e1[1];
        exact_scores<T, LPR, 1>(x, c, bias, a.scale, k1, a.d, a.vec, lane, e1);
        e[0] = e1[0];
      } else {
        exact_scores<T, LPR, 4>(x, c, bias, a.scale, k, a.d, a.vec, lane, e);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane == 0 && warp + 8 * i < a.cands) sh.exact[warp + 8 * i] = e[i];
    }
  } else {
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
    write_top(a, r, rank, mine, v, m, s, none, ls);
  }
}

// Many rows of few parts: a thread per row.  LL = 0: statistics only.
template <typename T, int LL>
__global__ void __launch_bounds__(256) k_join_rows(const JoinArgs a) {
  pdl_wait();
  constexpr int C = LL ? LL : 1;
  const int lane = threadIdx.x & 31;
  const long long r0 = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool live = r0 < a.rows;
  const long long r = live ? r0 : a.rows - 1, b = r / a.N;
  float m = kNegInf, s = 0.f, u = 0.f, tgt = kNegInf;
  for (int p = 0; p < a.parts; ++p) {
    const float4 q = __ldg(a.part + r * a.parts + p);
    join_stats(m, s, u, q.x, q.y, q.z);
    tgt = fmaxf(tgt, q.w);
  }
  const bool none = m == kNegInf && s == 0.f;
  const float ls = log2f(s);
  if (live) write_stats(a, r, m, s, u, tgt, none, ls);
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
      const float4 v4 = __ldg(pv + q);
      const int4 k4 = __ldg(pk + q);
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
    const float unit = bias ? 1.f : a.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < a.top) {
        a.top_ids[r * a.top + i] = hk[i];
        a.top_logp[r * a.top + i] = -at_least_0((ls - (hv[i] * unit - m)) * kLn2);
      }
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
        if (i < a.cands && rank < a.top) write_top(a, r, rank, hk[i], ev[i], m, s, none, ls);
      }
    }
  }
}

template <typename T, int LPR, int WPR, int LL>
int launch_join_as(const JoinArgs &j, cudaStream_t s) {
  const int per_block = WPR > 1 ? 1 : kJoinWarps * (32 / LPR);
  FK_CUDA(launch_pdl(k_join<T, LPR, WPR, LL>, dim3((unsigned)cdiv(j.rows, per_block)), dim3(32 * kJoinWarps), 0, s, j));
  return launched();
}

// A block per row while the rows alone do not fill the SMs; a thread per row
// where there are many, of few parts (604800 rows of 3 parts, top 4: 185 us against 246
// by 8 lanes a row); else as many lanes as there are candidates, at least 8.
template <typename T, int LL>
int launch_join_list(const JoinArgs &j, cudaStream_t s) {
  if (j.max_norm2) {
    FK_CUDA(cudaMemsetAsync(j.max_norm2, 0, (size_t)(j.rows / j.N) * sizeof(unsigned), s));
    const long long rows = j.rows / j.N * j.K;
    FK_CUDA(launch_pdl(k_max_norm<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const T *>(j.c), rows,
                       j.K, j.d, j.max_norm2));
    FK_TRY(launched());
  }
  if (j.rows > kJoinBlockRows && j.parts <= 8 && LL <= 16) {
    const dim3 grid((unsigned)cdiv(j.rows, 256));
    if (j.L) FK_CUDA(launch_pdl(k_join_rows<T, LL <= 16 ? LL : 16>, grid, dim3(256), 0, s, j));
    else FK_CUDA(launch_pdl(k_join_rows<T, 0>, grid, dim3(256), 0, s, j));
    return launched();
  }
  if (j.L && j.rows <= kJoinBlockRows) return launch_join_as<T, 32, 8, LL>(j, s);
  if (j.cands <= 8 && j.parts <= 64) return launch_join_as<T, 8, 1, LL>(j, s);
  if (j.cands <= 16) return launch_join_as<T, 16, 1, LL>(j, s);
  return launch_join_as<T, 32, 1, LL>(j, s);
}

template <typename T>
int launch_join_typed(const JoinArgs &j, cudaStream_t s) {
  if (j.L <= 4) return launch_join_list<T, 4>(j, s);
  if (j.L == 8) return launch_join_list<T, 8>(j, s);
  if (j.L <= 16) return j.L == 12 ? launch_join_list<T, 12>(j, s) : launch_join_list<T, 16>(j, s);
  return launch_join_list<T, 32>(j, s);
}

}  // namespace

int launch_join(const JoinArgs &j, int dtype, cudaStream_t s) {
  if (dtype == FK_F32) return launch_join_typed<float>(j, s);
  if (dtype == FK_BF16) return launch_join_typed<__nv_bfloat16>(j, s);
  return launch_join_typed<__half>(j, s);
}

}  // namespace soft
}  // namespace fk
