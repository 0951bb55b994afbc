// Tile engine of the soft assignment operators: a persistent, warp-specialised
// product of two 16-bit operands on tcgen05, whose epilogue is a template
// argument.  It serves
//   scores   S = X C^T        both operands with the contraction (d) contiguous,
//   dX       G C              C has its rows along the contraction ("MN-major"),
//   dC       G^T X            both operands have their rows along the contraction.
//
// One tile is 128 * CG rows by 256 columns: CG = 2 pairs two SMs on one tile
// (cta_group::2; each CTA stages its own 128 rows and half of the columns, so
// a K-block costs each SM 32 KB of operand traffic per 512 tensor cycles
// instead of the 48 KB of a lone CTA, which L2 cannot feed to all SMs).
//
//   warp 0      TMA producer (one thread): 64-wide K-blocks of both operands
//               into 128-byte-swizzled stages,
//   warp 1      one thread (of the pair's first CTA) issues tcgen05.mma,
//               M = 128 * CG, N = 256, K = 16; two 256-column accumulators in
//               TMEM let the next tile's products overlap this tile's epilogue,
//   warps 4-15  epilogue: three warps share each 32-row quadrant and take every
//               third 32 columns (the start moves from tile to tile, as 8 is
//               not a multiple of 3).
//
// fp32 operands come as three bf16 planes (hi, mid, lo: 8 + 8 + 8 significant
// bits) and the contraction runs over the six plane pairs whose product is
// above 2^-24 of the leading one, smallest of a segment first.  That costs 6 bf16 products,
// exactly the tensor time of three TF32 ones at half the rate, keeps fp32's
// range, and needs no second set of layouts (TF32 operands cannot be read
// MN-major).
//
// Work: a unit is one row tile against a run of consecutive column tiles (or
// one tile over a part of the contraction).  Units are numbered so that those
// in flight together cover one group of row tiles against the same columns:
// the columns' operand is read from HBM about once per group, and the group's
// rows stay in L2.
#pragma once

#include <type_traits>

#include "fk_sm100.cuh"

namespace fk {
namespace tile {

using namespace sm100;

constexpr int kRows = 128;   // rows of one CTA's tile
constexpr int kCols = 256;   // columns of a tile
constexpr int kK = 64;       // contraction elements per stage
// Four warpgroups: one for the producer and the MMA issuer (and two idle
// warps), three of epilogue.  The registers of a block launched with 128 a
// thread are split 56 / 152, or 32 / 160 for epilogues that keep segments and
// lists (128 * 4 = 56 + 3 * 152 = 32 + 3 * 160): those then spill little, at the
// price of spills around the producer's loads, which cost products without such
// an epilogue 6% (dX and dC of N 4096, K 65536, d 2048).
constexpr int kEpiWarps = 12;
constexpr int kFirstEpi = 4;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kLaunchRegs = 128;
template <int R>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

constexpr uint32_t kABytes = kRows * kK * 2;
// A chain of tcgen05 accumulations rounds towards zero at every step, which adds
// up to a bias of about steps / 2 half-units of the result (3e-6 of it at 2048
// terms).  Epilogues that ask for it (kSeg) get the contraction in segments,
// summed in registers with rounding to nearest: of 512 terms where fp32 results
// hang on them, of 4096 (a bias of 2.6e-5 at most) where the result is rounded
// to 16 bits.  One chain of 40000 terms was off by 1.3e-4, a quarter of fp16's
// half step; segments of 1024 cost products of a training step 5%, these 1%
// (N 4096, K 65536, d 2048).
constexpr int kSegBlocks = 8, kLongSegBlocks = 64;
constexpr int kMaxStages = 8;
constexpr int kCtrlBytes = 256;  // barriers, TMEM address, abort flag

template <int CG>
struct Geo {
  static constexpr uint32_t kBBytes = kCols / CG * kK * 2;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
};

struct Plan {
  int cg;           // CTAs per tile
  int units;        // B * ksplits * runs * row_tiles
  int row_tiles;    // tiles of 128 * CG rows
  int col_tiles;
  int runs;         // column runs per row tile
  int ksplits;      // parts of the contraction
  int group;        // row tiles per group
  int kblocks;      // 64-wide blocks of one plane pair
  int pairs;        // of planes: 1, 2 (A in two parts), or 6 for fp32
  int planes_a, planes_b;  // 1, 2 or 3
  int stages;
  uint32_t idesc;
};

struct Unit {
  int b, rt, ct0, ct1, k0, k1, run, ks;
};

__host__ __device__ __forceinline__ Unit unit_of(const Plan &p, int u) {
  Unit w;
  const int per_b = p.ksplits * p.runs * p.row_tiles;
  w.b = u / per_b;
  int r = u - w.b * per_b;
  const int full = p.ksplits * p.runs * p.group;
  const int g = r / full;
  r -= g * full;
  const int rows = p.row_tiles - g * p.group < p.group ? p.row_tiles - g * p.group : p.group;
  const int q = r / rows;
  w.rt = g * p.group + (r - q * rows);
  w.ks = q / p.runs;
  w.run = q - w.ks * p.runs;
  w.ct0 = (int)((long long)w.run * p.col_tiles / p.runs);
  w.ct1 = (int)((long long)(w.run + 1) * p.col_tiles / p.runs);
  const long long kt = (long long)p.pairs * p.kblocks;
  w.k0 = (int)(w.ks * kt / p.ksplits);
  w.k1 = (int)((w.ks + 1) * kt / p.ksplits);
  return w;
}

// The plane pair of a contraction step, smallest products of a group of K-blocks first.
__device__ __forceinline__ void pair_planes(int pairs, int pair, int &pa, int &pb) {
  if (pairs < 6) {
    pa = pairs - 1 - pair;
    pb = 0;
    return;
  }
  // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
  pa = (0x001012 >> (4 * pair)) & 15;
  pb = (0x010210 >> (4 * pair)) & 15;
}

// Descriptor of an operand whose contraction index is the row of the tile:
// blocks of 64 columns (128 bytes, 128-byte swizzle) by 64 rows; 8-row groups
// 1024 bytes apart, the next 64 columns one block (8 KB) further.  16 rows
// (one MMA step) are 2048 bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
  uint64_t desc = 0;
  desc |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  desc |= (uint64_t)(8192u >> 4) << 16;
  desc |= (uint64_t)(1024u >> 4) << 32;
  desc |= (uint64_t)1u << 46;
  desc |= (uint64_t)2u << 61;
  return desc;
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 1) {
    mma_f16(d, a, b, idesc, acc);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  }
}

// Commit of the MMAs issued so far: one arrival on `bar` of every CTA of the pair.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            bar),
        "h"((uint16_t)3)
        : "memory");
  }
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Tiled load whose bytes are counted on a barrier of the pair's first CTA
// (bar: a shared::cluster address).
template <int CG>
__device__ __forceinline__ void load_3d(const CUtensorMap *map, uint32_t dst, uint32_t bar, int c0, int c1, int c2) {
  if constexpr (CG == 1) {
    tma_load_3d(map, dst, bar, c0, c1, c2);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  }
}

template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t dst, uint32_t n) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, n);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(n) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t addr, uint32_t n) {
  if constexpr (CG == 1) tmem_dealloc(addr, n);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(n) : "memory");
}

// Waits for this thread's TMEM loads; the registers they fill pass through, so
// that no use of them can be moved ahead of the wait.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// All lanes return the same verdict of a wait that lane 0 polls.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *err,
                                          int lane) {
  int ok = 1;
  if (lane == 0) ok = mbar_wait_spin(bar, parity, abort_flag, err);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();  // the exchange orders no memory: the wait does, and this hands it on
  return ok != 0;
}

// What an epilogue sees.  Epi provides
//   struct Args                    kernel argument
//   static constexpr int kSeg      K-blocks of a segment of the contraction, summed in registers; 0: one chain
//   static constexpr int kRegs     registers of an epilogue thread, 152 or 160
//   begin(const Unit &, row0)      before the unit's first tile
//   skip(column)                   warp-uniform: nothing to do from this column on
//   prepare(column, stride)        before the wait for a tile's products: the warp's
//                                  32-column chunks start at column, + stride, ...
//   chunk(32 values, column, i)    the row's values of the warp's i-th chunk
//   end(const Unit &)              after the unit's last tile
// and is constructed per thread with (args, lane, row in CTA tile, warp of the
// quadrant, shared memory).
template <int CG, bool A_MN, bool B_MN, class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    k_tiles(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
            const __grid_constant__ Plan p, const __grid_constant__ typename Epi::Args ea, int *err) {
  extern __shared__ uint8_t smem_raw[];
  using G = Geo<CG>;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *gen = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t ctrl = base + p.stages * G::kStageBytes;
  uint8_t *ctrl_gen = gen + p.stages * G::kStageBytes;
  auto full = [&](int s) { return ctrl + 8u * s; };
  auto empty = [&](int s) { return ctrl + 64u + 8u * s; };
  auto tfull = [&](int i) { return ctrl + 128u + 8u * i; };
  auto tempty = [&](int i) { return ctrl + 144u + 8u * i; };
  const uint32_t tmem_slot = ctrl + 160u;
  volatile int *abort_flag = reinterpret_cast<int *>(ctrl_gen + 164);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cta_rank();
  const int worker = blockIdx.x / CG, workers = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), kEpiWarps * CG);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&ta);
    prefetch_tensormap(&tb);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the pair's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctrl_gen + 160);
  pdl_wait();
  pdl_trigger();

  if (warp < kFirstEpi) {
  give_registers<4 * kLaunchRegs - 3 * Epi::kRegs>();
  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 1;  // parity of the stage's last release
      bool ok = true;
      for (int u = worker; u < p.units && ok; u += workers) {
        const Unit w = unit_of(p, u);
        const int arow = (w.rt * CG + (int)rank) * kRows;
        for (int ct = w.ct0; ct < w.ct1 && ok; ++ct) {
          const int bcol = ct * kCols + (int)rank * (kCols / CG);
          // kSegBlocks K-blocks of every plane pair, then the next kSegBlocks: a
          // plane is read again while it is in L2 (fp32 training, N 14, K 61507,
          // d 2670: 1890 us against 1970 with a pair's whole contraction at a time)
          int g0 = w.k0 / (kSegBlocks * p.pairs);
          const int at = w.k0 - g0 * (kSegBlocks * p.pairs);
          g0 *= kSegBlocks;
          int gend = min(g0 + kSegBlocks, p.kblocks), pair = at / (gend - g0), kb = g0 + at - pair * (gend - g0);
          int pa, pb;
          pair_planes(p.pairs, pair, pa, pb);
          pa += w.b * p.planes_a;
          pb += w.b * p.planes_b;
          for (int k = w.k0; k < w.k1; ++k, ++it) {
            if (!mbar_wait_spin(empty(s), ph, abort_flag, err)) { ok = false; break; }
            const uint32_t sa = base + s * G::kStageBytes, sb = sa + kABytes;
            const uint32_t bar = CG == 1 ? full(s) : map_to_cta(full(s), 0);
            if (rank == 0) mbar_arrive_expect_tx(full(s), G::kStageBytes * CG);
            if constexpr (A_MN) {
#pragma unroll
              for (int i = 0; i < kRows / 64; ++i)
                load_3d<CG>(&ta, sa + i * 8192u, bar, arow + i * 64, kb * kK, pa);
            } else {
              load_3d<CG>(&ta, sa, bar, kb * kK, arow, pa);
            }
            if constexpr (B_MN) {
#pragma unroll
              for (int i = 0; i < kCols / CG / 64; ++i)
                load_3d<CG>(&tb, sb + i * 8192u, bar, bcol + i * 64, kb * kK, pb);
            } else {
              load_3d<CG>(&tb, sb, bar, kb * kK, bcol, pb);
            }
            if (++kb == gend) {
              if (++pair == p.pairs) {
                pair = 0;
                g0 = gend;
                gend = min(g0 + kSegBlocks, p.kblocks);
              }
              kb = g0;
              pair_planes(p.pairs, pair, pa, pb);
              pa += w.b * p.planes_a;
              pb += w.b * p.planes_b;
            }
            if (++s == p.stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
      }
      // leave only when the issued copies have landed: every stage was handed
      // back by the MMA (bounded; after an abort the copies get a millisecond)
      if (ok) {
        const uint32_t n = it < (uint32_t)p.stages ? it : (uint32_t)p.stages;
        for (uint32_t j = it - n; j < it; ++j)
          if (!mbar_wait_spin(empty(j % p.stages), (j / p.stages) & 1, abort_flag, err)) { ok = false; break; }
      }
      if (!ok) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {}
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      uint32_t n = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = worker; u < p.units && ok; u += workers) {
        const Unit w = unit_of(p, u);
        for (int ct = w.ct0; ct < w.ct1 && ok; ++ct) {
          for (int ks = w.k0; ks < w.k1 && ok; ++n) {
            const int ke = Epi::kSeg && w.k1 - ks > Epi::kSeg ? ks + Epi::kSeg : w.k1;
            const uint32_t buf = n & 1;
            if (!mbar_wait_spin(tempty(buf), ((n >> 1) & 1) ^ 1, abort_flag, err)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d = tmem + buf * kCols;
            for (int k = ks; k < ke; ++k) {
              if (!mbar_wait_spin(full(s), ph, abort_flag, err)) { ok = false; break; }
              tc_fence_after();
              const uint32_t sa = base + s * G::kStageBytes, sb = sa + kABytes;
#pragma unroll
              for (int kk = 0; kk < kK / 16; ++kk) {
                const uint64_t da = A_MN ? desc_mn_sw128(sa + kk * 2048u) : desc_k_sw128(sa + kk * 32u);
                const uint64_t db = B_MN ? desc_mn_sw128(sb + kk * 2048u) : desc_k_sw128(sb + kk * 32u);
                mma<CG>(d, da, db, p.idesc, k > ks || kk > 0);
              }
              commit<CG>(empty(s));
              if (++s == p.stages) {
                s = 0;
                ph ^= 1;
              }
            }
            if (ok) commit<CG>(tfull(buf));
            ks = ke;
          }
        }
      }
    }
  }
  } else {
    take_registers<Epi::kRegs>();
    const int quad = warp & 3, third = (warp - kFirstEpi) >> 2;
    Epi epi(ea, lane, quad * 32 + lane, third, ctrl_gen + kCtrlBytes);
    uint32_t n = 0;
    bool ok = true;
    auto release = [&](uint32_t buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1 || rank == 0) mbar_arrive(tempty(buf));
        else arrive_cluster(map_to_cta(tempty(buf), 0));
      }
    };
    for (int u = worker; u < p.units && ok; u += workers) {
      const Unit w = unit_of(p, u);
      epi.begin(w, (w.rt * CG + (int)rank) * kRows);
      for (int ct = w.ct0; ct < w.ct1 && ok; ++ct) {
        const int first = (third + ct) % 3 * 32;
        const long long col0 = (long long)ct * kCols + first;
        const uint32_t lanes = tmem + first + ((uint32_t)(quad * 32) << 16);
        epi.prepare(col0, 96);
        if constexpr (Epi::kSeg > 0) {
          float sum[3][32];
          auto segment = [&](auto add) {
            const uint32_t buf = n & 1;
            if (!warp_wait(tfull(buf), (n >> 1) & 1, abort_flag, err, lane)) return false;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              if (first + 96 * i < kCols && !epi.skip(col0 + 96 * i)) {
                if constexpr (decltype(add)::value) {
                  uint32_t acc[32];
                  tmem_ld_32x32b_x32(lanes + buf * kCols + 96 * i, acc);
                  wait_ld(acc);
#pragma unroll
                  for (int j = 0; j < 32; j += 2) {
                    const float2 v = __fadd2_rn(make_float2(sum[i][j], sum[i][j + 1]),
                                                make_float2(__uint_as_float(acc[j]), __uint_as_float(acc[j + 1])));
                    sum[i][j] = v.x;
                    sum[i][j + 1] = v.y;
                  }
                } else {
                  tmem_ld_32x32b_x32(lanes + buf * kCols + 96 * i, reinterpret_cast<uint32_t(&)[32]>(sum[i]));
                }
              }
            }
            if constexpr (!decltype(add)::value) {
#pragma unroll
              for (int i = 0; i < 3; ++i) wait_ld(reinterpret_cast<uint32_t(&)[32]>(sum[i]));
            }
            release(buf);
            ++n;
            return true;
          };
          ok = segment(std::false_type{});
          for (int ks = w.k0 + Epi::kSeg; ks < w.k1 && ok; ks += Epi::kSeg) ok = segment(std::true_type{});
          if (ok) {
            // one copy of the epilogue's code: the sums move up instead
#pragma unroll 1
            for (int i = 0; first + 96 * i < kCols; ++i) {
              if (epi.skip(col0 + 96 * i)) break;
              epi.chunk(sum[0], col0 + 96 * i, i);
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[q][j] = sum[q + 1][j];
            }
          }
        } else {
          const uint32_t buf = n & 1;
          if (!warp_wait(tfull(buf), (n >> 1) & 1, abort_flag, err, lane)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; first + 96 * i < kCols; ++i) {
            if (epi.skip(col0 + 96 * i)) break;
            float acc[32];
            tmem_ld_32x32b_x32(lanes + buf * kCols + 96 * i, reinterpret_cast<uint32_t(&)[32]>(acc));
            wait_ld(reinterpret_cast<uint32_t(&)[32]>(acc));
            epi.chunk(acc, col0 + 96 * i, i);
            __syncwarp();  // the next load is warp-wide
          }
          release(buf);
          ++n;
        }
      }
      if (ok) epi.end(w);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem, 512);
  }
}

}  // namespace tile
}  // namespace fk
