// The product of two packed 4-bit matrices (fp4.cuh) on SM pairs, for more than
// a few rows:
//   C[m][n] = ((sum_k a*sa * b*sb) * ga[m]) * gb[n]
// with the block scales applied by the block-scaled MMA (tcgen05.mma
// kind::mxf4nvf4, K = 64 an instruction, fp32 accumulation in tensor memory) and
// the row scales of block 16 in the epilogue.
//
// Tiles that do not fill a last round of all pairs are cut into pieces 128 or 64
// columns wide where that gives every pair one (4096 x 4096 x 11008: 256 tiles on
// 76 pairs are 3 rounds and 28 tiles, run as 56 pieces).
//
// Cluster of 2 CTAs per 256 x 256 tile of C, persistent over the tiles, 352
// threads each. A tile's columns are two parts of 128, each one 128-row tile of B
// of which either CTA holds 64 rows (twice as many MMAs of half the width run at
// the same rate, and a part can start by itself).
//  * warps 9 and 10: copy this CTA's 128 rows of A and its halves of B's two row
//    tiles (256 columns of K a stage: 16 KB of codes each), the scales of its rows
//    of A and those of all 256 rows of B into a ring, a warp for each operand: one
//    warp issuing all six copies of a stage was late with them (4096 x 4096 x
//    11008, block 32: 58.5 us with one, 53.2 with two). The packed layout is the
//    MMA's own, so every copy is one contiguous run or eight; a tensor map
//    describes it as a plain matrix only because tensor copies can complete on the
//    even CTA's barrier.
//  * warp 8 of the even CTA: moves each 128 columns' scales to tensor memory
//    (tcgen05.cp, both CTAs at once) and issues the pair MMAs.
//  * warps 0-7: one row and 128 columns a thread; scale, round, stage 32 rows x
//    128 bytes in shared memory and store the box by TMA (row pitches that TMA
//    cannot take are stored from the staged rows by the warp).
// Tensor memory: 512 columns cannot hold two 256-column accumulators and the
// scales, so the accumulators of even and odd tiles overlap in 64 columns
// (0..255 and 192..447; the scales at 448). The epilogue empties those 64 first;
// until then the next tile runs its first stages on the part that is free.
//
// What bounds it: the MMA with K = 64 alone sustains about 9.6 PFLOP/s here
// (124 cycles for 256 x 256 x 64). 8192 x 11008 x 4096 bf16 output, block 32: 106 to
// 112 us from run to run (7.0 to 6.6 PFLOP/s), of which the stores of C cost 15 us
// or more (91 us without them): their bursts delay the loads, and five stages (2500
// cycles) cannot ride that out. So the stores are spread over the next tile's time
// (4096 x 11008 x 4096 without this and the early start 62.8 us in blocks of 16 and
// 59.4 in blocks of 32; now 60.3 and 56.0). B shared by two pairs through
// multicast in clusters of four made no pair faster and leaves 8 of 152 SMs idle
// (121 us); smaller stages are bound by the issuing warp (145 us).
// Every wait is bounded (common.cuh).
#include "chain.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "gemm_fp4.cuh"
#include "kernels.h"
#include "tma.h"

#include <algorithm>
#include <mutex>

namespace qmm {
namespace gfp4 {
namespace pair {

constexpr int NEW = 8;
constexpr int NT = NEW * 32 + 96;   // + MMA warp + two producer warps
constexpr int NS = 5;
constexpr int STAGE_KT = 2;                       // 128-column tiles of K a stage
constexpr int CODE_BYTES = STAGE_KT * 8192;       // one operand's codes a stage and CTA
constexpr int PART_BYTES = CODE_BYTES / 2;        // a CTA's codes of 128 columns of C a stage: 64 rows of B
constexpr long long kPaceLimit = 100000;          // cycles that the stores of a tile may be spread over
constexpr int AHEAD = 3;                          // stages that a tile may start on half its columns
constexpr int STG_BYTES = 32 * 128;               // a warp's staged rows
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC1 = 192;                    // first column of odd tiles' accumulator
constexpr uint32_t SF_COL = 448;                  // two buffers of 24 columns: A's 8, B's 16

struct Shared {
  uint64_t full[NS], empty[NS];
  uint64_t acc_full[2];   // the pair's commit, per tile parity
  uint64_t acc_free;      // even CTA: the columns shared with the next tile are read; one arrival per epilogue warp
  uint64_t acc_done[2];   // of both CTAs and tile. All columns are, per tile parity
  uint64_t teardown;
  uint32_t tmem_base;
  int abort_flag;
  float gb[NEW][64];      // per epilogue warp, the column scales of the 64 columns it works on (block 16)
};

// The tiles of a launch: `full` of them 256 columns wide, dealt out in turn, then
// the rest in pieces of 256 / cut columns, one to a cluster.
constexpr int kBand = 8;
struct Sched {
  int full, cut, pieces, m_tiles;
};
struct Work {
  int mt, nt;    // tile
  int piece;     // of the tile's columns (0 for a whole tile)
  int width;     // columns: 256, 128 or 64
};
__device__ __forceinline__ int work_count(const Sched& sc, int cid, int ncl) {
  return (cid < sc.full ? (sc.full - cid + ncl - 1) / ncl : 0) + (cid < sc.pieces ? 1 : 0);
}
__device__ __forceinline__ Work work_at(const Sched& sc, int i, int cid, int ncl, int n_tiles) {
  Work w;
  int tile = cid + i * ncl;
  w.piece = 0;
  w.width = 256;
  if (tile >= sc.full) {
    tile = sc.full + cid / sc.cut;
    w.piece = cid - cid / sc.cut * sc.cut;
    w.width = 256 / sc.cut;
  }
  // bands of kBand rows of tiles, down the columns of a band
  const int band = tile / (kBand * n_tiles), in = tile - band * kBand * n_tiles;
  const int rows = min(kBand, sc.m_tiles - band * kBand);
  w.nt = in / rows;
  w.mt = band * kBand + in - w.nt * rows;
  return w;
}

enum : unsigned {
  SITE_EMPTY = 0x510, SITE_FULL = 0x511, SITE_ACC_FULL = 0x512, SITE_ACC_FREE = 0x513, SITE_TEARDOWN = 0x514,
  SITE_FINAL = 0x515, SITE_ACC_DONE = 0x516
};

// Tensor copies that complete on the even CTA's barrier, issued by the lane whose
// `on` is set (the producer warps run converged, as the issuer does).
__device__ __forceinline__ void load_pair(uint32_t dst, const void* tmap, int row, uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];\n\t}" ::"r"(dst),
      "l"(tmap), "r"(0), "r"(row), "r"(bar), "r"(on)
      : "memory");
}
__device__ __forceinline__ void load_pair_3d(uint32_t dst, const void* tmap, int chunk, int part, uint32_t bar,
                                             uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(tmap), "r"(0), "r"(chunk), "r"(part), "r"(bar), "r"(on)
      : "memory");
}
__device__ __forceinline__ void expect_on(uint64_t* bar, uint32_t bytes, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(on)
      : "memory");
}

// whether the phase has completed, without waiting
__device__ __forceinline__ bool mbar_test_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

template <int BLOCK>
struct Cfg {
  static constexpr int ATOMS = BLOCK == 16 ? 2 : 1;            // scale atoms per 128 columns
  static constexpr int SF_BYTES = STAGE_KT * ATOMS * 512;      // 128 rows' scales a stage
  static constexpr int STAGE = 2 * CODE_BYTES + 3 * SF_BYTES;  // A, B, A's scales, B's two halves
  static constexpr size_t SMEM = (size_t)NS * STAGE + NEW * STG_BYTES + sizeof(Shared) + 1024;
};
static_assert(Cfg<16>::SMEM <= 232448, "shared memory per CTA");

// The issuing warp's place in the ring of stages and scale buffers.
struct Issuer {
  uint32_t s16, tb, on;   // ring base / 16, tensor memory base, this lane issues
  int slot;
  uint32_t phase, buf;

  __device__ __forceinline__ void advance() {
    if (++slot == NS) {
      slot = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ bool wait_full(Shared& sm, unsigned* err) {
    const bool ok = mbar_wait(&sm.full[slot], phase, &sm.abort_flag, err, SITE_FULL);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    return true;
  }

  // The stage at `slot` (n tiles of 128 columns of K) for parts P0 .. P1 - 1 of the
  // tile's columns: a tile of 256 has two parts of 128, a piece is one part of
  // WIDTH. odd: tensor memory columns by which a piece's scales of B start after
  // their atom (an odd piece of 64 columns is the second half of its 128 rows).
  template <int BLOCK, int WIDTH, int P0, int P1>
  __device__ __forceinline__ void stage(int n, uint32_t tacc, uint32_t odd, uint32_t accumulate) {
    using C = Cfg<BLOCK>;
    constexpr int ATOMS = C::ATOMS, PW = WIDTH == 64 ? 64 : 128;   // a part's columns
    constexpr uint32_t id0 = idesc_fp4(256, PW, BLOCK == 32, 0), id1 = idesc_fp4(256, PW, BLOCK == 32, 2);
    constexpr uint32_t b_ch = PW / 2;                 // a CTA's rows of a part of B: a chunk's bytes / 16
    constexpr uint32_t b_lo = b_ch << 16;
    const uint32_t a = s16 + (uint32_t)slot * (C::STAGE >> 4), b = a + (CODE_BYTES >> 4);
    const uint32_t fa = b + (CODE_BYTES >> 4), fb = fa + (C::SF_BYTES >> 4);
#pragma unroll
    for (int k = 0; k < STAGE_KT; ++k) {
      if (k > 0 && n == 1) break;
      const uint32_t sa = tb + SF_COL + buf, sb = sa + 8u;
      buf ^= 24u;
#pragma unroll
      for (int i = 0; i < ATOMS; ++i) {
        cp_scales_pair(sa + i * 4, fa + (k * ATOMS + i) * 32, on);
#pragma unroll
        for (int h = P0; h < P1; ++h)
          cp_scales_pair(sb + (h * ATOMS + i) * 4, fb + h * (C::SF_BYTES >> 4) + (k * ATOMS + i) * 32, on);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)   // 64 columns of K each
#pragma unroll
        for (int h = P0; h < P1; ++h)
          mma_fp4_pair<BLOCK>(tacc + h * 128, a + (uint32_t)(k * 512 + j * 256) + kDescLo,
                              b + h * (PART_BYTES >> 4) + (uint32_t)(k * 4 + j * 2) * b_ch + b_lo,
                              (BLOCK == 32 && j) ? id1 : id0, sa + (BLOCK == 16 ? j * 4 : 0),
                              sb + (h * ATOMS + (BLOCK == 16 ? j : 0)) * 4 + (WIDTH == 64 ? odd : 0u),
                              (k > 0 || j > 0) ? 1u : accumulate, on);
    }
  }

  // Stages [from, stages) of a tile or piece. False if a wait ran out.
  template <int BLOCK, int WIDTH>
  __device__ __forceinline__ bool run(Shared& sm, unsigned* err, int kt, int from, uint32_t tacc, uint32_t odd) {
    for (int left = kt - from * STAGE_KT; left > 0; left -= STAGE_KT) {
      if (!wait_full(sm, err)) return false;
      stage<BLOCK, WIDTH, 0, WIDTH == 256 ? 2 : 1>(left, tacc, odd, left == kt ? 0u : 1u);
      commit_pair_on(&sm.empty[slot], on);
      advance();
    }
    return true;
  }

  // Part FREE of up to AHEAD first stages, until the previous tile's columns are
  // drained; then the other part of the same stages. Returns their number, -1 if a
  // wait ran out.
  template <int BLOCK, int FREE>
  __device__ __forceinline__ int start(Shared& sm, unsigned* err, int kt, uint32_t tacc, uint32_t parity) {
    const int slot0 = slot;
    const uint32_t phase0 = phase;
    int ahead = 0;
    while (ahead < AHEAD && ahead * STAGE_KT < kt) {
      if (__all_sync(0xffffffffu, mbar_test_cluster(&sm.acc_free, parity))) break;
      if (!wait_full(sm, err)) return -1;
      stage<BLOCK, 256, FREE, FREE + 1>(kt - ahead * STAGE_KT, tacc, 0u, ahead ? 1u : 0u);
      advance();
      ++ahead;
    }
    if (!__all_sync(0xffffffffu, mbar_wait_cluster(&sm.acc_free, parity, &sm.abort_flag, err, SITE_ACC_FREE))) return -1;
    tc_fence_after();
    slot = slot0;
    phase = phase0;
    for (int i = 0; i < ahead; ++i) {
      stage<BLOCK, 256, 1 - FREE, 2 - FREE>(kt - i * STAGE_KT, tacc, 0u, i ? 1u : 0u);
      commit_pair_on(&sm.empty[slot], on);
      advance();
    }
    return ahead;
  }
};

template <int BLOCK>
__global__ void __launch_bounds__(NT, 1)
    gemm_fp4_pair_kernel(const GemmFp4Args p, const int tma_c, const Sched sc, const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmBP,
                         const __grid_constant__ CUtensorMap tmSA,
                         const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmC) {
  using C = Cfg<BLOCK>;
  constexpr int ATOMS = C::ATOMS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const uint32_t stg_base = sbase + NS * C::STAGE;
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw + (sbase - raw) + NS * C::STAGE + NEW * STG_BYTES);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t rank = cluster_ctarank();
  const int cid = (int)cluster_id_x(), ncl = (int)nclusters_x();
  const Fp4Layout LA(p.M, p.K, BLOCK), LB(p.N, p.K, BLOCK);
  const int n_tiles = (int)((p.N + 255) / 256);
  const int my_tiles = work_count(sc, cid, ncl);
  const int kt = (int)LA.kt;

  if (t == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.acc_full[0], 1);
    mbar_init(&sm.acc_full[1], 1);
    mbar_init(&sm.acc_free, 2 * NEW);
    mbar_init(&sm.acc_done[0], 2 * NEW);
    mbar_init(&sm.acc_done[1], 2 * NEW);
    mbar_init(&sm.teardown, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == NEW) {
    tmem_alloc_pair(&sm.tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  chain_wait();   // what is above ran under the call before

  if (warp == NEW) {
    // ---------------- pair MMA issuer (even CTA, the warp converged) ----------------
    if (rank == 0) {
      const uint32_t on = elect_one();
      const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
      Issuer ring{desc_addr(sbase), tb, on, 0, 0u, 0u};
      // broadcast from one lane, so that the compiler sees the warp's control flow is uniform
      const int cid_u = __shfl_sync(0xffffffffu, cid, 0), tiles_u = __shfl_sync(0xffffffffu, my_tiles, 0);
      bool ok = true;
      for (int tl = 0; tl < tiles_u && ok; ++tl) {
        const uint32_t tacc = tb + ((tl & 1) ? ACC1 : 0u);
        const Work wk = work_at(sc, tl, cid_u, ncl, n_tiles);
        const int width = __shfl_sync(0xffffffffu, wk.width, 0);
        const uint32_t odd = __shfl_sync(0xffffffffu, wk.piece & 1, 0) ? 2u : 0u;
        // this accumulator's last tile is drained; the previous tile's columns
        // (shared by an odd tile's first part, an even tile's second) are soon
        int begun = 0;
        if (tl > 1) {
          ok = mbar_wait_cluster(&sm.acc_done[tl & 1], (uint32_t)(((tl >> 1) - 1) & 1), &sm.abort_flag, p.err,
                                 SITE_ACC_DONE);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        tc_fence_after();
        if (tl > 0 && width == 256) {
          begun = (tl & 1) ? ring.template start<BLOCK, 1>(sm, p.err, kt, tacc, 0u)
                           : ring.template start<BLOCK, 0>(sm, p.err, kt, tacc, 1u);
          ok = begun >= 0;
          if (!ok) break;
        } else if (tl > 0) {
          ok = mbar_wait_cluster(&sm.acc_free, (uint32_t)((tl - 1) & 1), &sm.abort_flag, p.err, SITE_ACC_FREE);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        if (width == 256) ok = ring.template run<BLOCK, 256>(sm, p.err, kt, begun, tacc, odd);
        else if (width == 128) ok = ring.template run<BLOCK, 128>(sm, p.err, kt, 0, tacc, odd);
        else ok = ring.template run<BLOCK, 64>(sm, p.err, kt, 0, tacc, odd);
        if (!ok) break;
        commit_pair_on(&sm.acc_full[tl & 1], on);
      }
    }
    __syncwarp();
  } else if (warp > NEW) {
    // ---------------- producers (both CTAs): warp 9 A, warp 10 B ----------------
    const bool is_a = warp == NEW + 1;
    const uint32_t on = elect_one();
    if (on) {
      prefetch_tmap(is_a ? &tmA : &tmB);
      prefetch_tmap(is_a ? &tmSA : &tmSB);
      if (!is_a && sc.cut > 2) prefetch_tmap(&tmBP);
    }
    const uint32_t full0 = mapa_shared(smem_u32(&sm.full[0]), 0);
    const int cid_u = __shfl_sync(0xffffffffu, cid, 0), tiles_u = __shfl_sync(0xffffffffu, my_tiles, 0);
    const int rank_u = __shfl_sync(0xffffffffu, (int)rank, 0);
    const uint32_t expect = rank_u == 0 && is_a ? on : 0u;
    int g = 0, slot = 0;
    uint32_t phase = 1u;   // a fresh slot is empty: the first round's waits pass
    bool ok = true;
    for (int tl = 0; tl < tiles_u && ok; ++tl) {
      const Work wk = work_at(sc, tl, cid_u, ncl, n_tiles);
      const int width = __shfl_sync(0xffffffffu, wk.width, 0);
      const bool whole = width == 256;
      // row tiles of this CTA (past the matrix: the last one again; its results are not stored)
      const int last = (int)LB.rt - 1;
      const int ra = min(2 * wk.mt + rank_u, (int)LA.rt - 1);
      // row tiles of B: both of a whole tile, a piece's one
      const int rb0 = min(2 * wk.nt + (width == 64 ? wk.piece >> 1 : wk.piece), last);
      const int rb1 = min(2 * wk.nt + 1, last);
      // the CTA's part of a row tile: a half, of a piece of 64 columns a quarter
      const int part = width >= 128 ? rank_u : 2 * (wk.piece & 1) + rank_u;
      const uint32_t bytes =
          2u * (whole ? (uint32_t)C::STAGE : (uint32_t)(CODE_BYTES + width * 32 * STAGE_KT + 2 * C::SF_BYTES));
      const int f0 = is_a ? ra * kt : rb0 * kt, f1 = rb1 * kt;
      for (int s = 0; s < kt; s += STAGE_KT, ++g) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[slot], phase, &sm.abort_flag, p.err, SITE_EMPTY));
        if (!ok) break;
        const uint32_t bar = full0 + (uint32_t)slot * 8u;
        const uint32_t dst = sbase + (uint32_t)slot * C::STAGE, sf = dst + 2 * CODE_BYTES;
        expect_on(&sm.full[slot], bytes, expect);
        // a stage that reaches past its row tile copies bytes that no MMA reads
        if (is_a) {
          load_pair(dst, &tmA, (f0 + s) * 8, bar, on);
          load_pair(sf, &tmSA, (f0 + s) * ATOMS, bar, on);
        } else if (whole) {
          load_pair_3d(dst + CODE_BYTES, &tmB, (f0 + s) * 4, part, bar, on);
          load_pair_3d(dst + CODE_BYTES + PART_BYTES, &tmB, (f1 + s) * 4, part, bar, on);
          load_pair(sf + C::SF_BYTES, &tmSB, (f0 + s) * ATOMS, bar, on);
          load_pair(sf + 2 * C::SF_BYTES, &tmSB, (f1 + s) * ATOMS, bar, on);
        } else {
          load_pair_3d(dst + CODE_BYTES, width == 128 ? &tmB : &tmBP, (f0 + s) * 4, part, bar, on);
          load_pair(sf + C::SF_BYTES, &tmSB, (f0 + s) * ATOMS, bar, on);
        }
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    // the even CTA's barriers count both CTAs' bytes: once the last stages'
    // phases complete, no copy of either CTA is in flight
    if (rank == 0 && is_a)
      for (int j = (g > NS ? g - NS : 0); j < g; ++j)
        mbar_wait_cluster(&sm.full[j % NS], (uint32_t)((j / NS) & 1), nullptr, p.err, SITE_FINAL);
    __syncwarp();
  } else {
    // ---------------- epilogue ----------------
    const int q = warp & 3, h = warp >> 2;
    const uint32_t free0 = mapa_shared(smem_u32(&sm.acc_free), 0);
    const uint32_t done0 = mapa_shared(smem_u32(&sm.acc_done[0]), 0);
    const uint32_t stg = stg_base + (uint32_t)warp * STG_BYTES;
    const float* rows_a = reinterpret_cast<const float*>(p.A + LA.row_off());
    const float* rows_b = reinterpret_cast<const float*>(p.B + LB.row_off());
    long long last = 0;
    for (int tl = 0; tl < my_tiles; ++tl) {
      const Work wk = work_at(sc, tl, cid, ncl, n_tiles);
      const long long row0 = (long long)wk.mt * 256 + rank * 128 + q * 32;
      // this warp's columns: half of a whole tile's or of 128; all 64 of the narrowest
      const int hc = wk.width == 256 ? 128 : 64;
      const long long col0 = (long long)wk.nt * 256 + wk.piece * wk.width + h * hc;
      const int units = wk.width == 256 ? 2 : (wk.width == 128 || h == 0) ? 1 : 0;
      float ga = 1.f, gb[4] = {};   // this lane's row scale; column scales lane, lane + 32, ...
      if (BLOCK == 16) {
        if (row0 + lane < p.M) ga = __ldg(rows_a + row0 + lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col0 + i * 32 + lane < p.N) gb[i] = __ldg(rows_b + col0 + i * 32 + lane);
      }
      if (!mbar_wait_cluster(&sm.acc_full[tl & 1], (uint32_t)((tl >> 1) & 1), &sm.abort_flag, p.err, SITE_ACC_FULL))
        break;
      // the time that the next tile will take, if that is a whole one too: as this one
      // did (rows stored by the warps are spread as it is)
      const long long now = clock64();
      const bool paced = tma_c && tl > 0 && tl + 1 < my_tiles && work_at(sc, tl + 1, cid, ncl, n_tiles).width == 256;
      const long long period = paced ? min(now - last, kPaceLimit) : 0;
      last = now;
      tc_fence_after();
      const uint32_t tacc = tbase + ((uint32_t)(q * 32) << 16) + ((tl & 1) ? ACC1 : 0u) + (uint32_t)(h * hc);
      // even tiles share columns 192..255 with the next accumulator, odd ones 0..63
      const int first = (tl & 1) || units < 2 ? 0 : 1;
      const uint32_t done = done0 + (uint32_t)(tl & 1) * 8u;
      const bool shares = units == 2 && h == ((tl & 1) ? 0 : 1);   // (a piece is the last of its cluster)
      if (tl == my_tiles - 1) chain_release();
      if (!shares) {
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_cta(free0);
        if (lane == 0 && units == 0) mbar_arrive_remote_cta(done);
      }
#pragma unroll 1
      for (int u = 0; u < units; ++u) {
        const int unit = u ^ first;   // 64 columns
        uint32_t acc[2][32];
        tmem_ld32x2(tacc + unit * 64, acc[0], tacc + unit * 64 + 32, acc[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && shares && u == 0) mbar_arrive_remote_cta(free0);
        if (lane == 0 && u == units - 1) mbar_arrive_remote_cta(done);
        if (period > 0) {   // quarters of the next tile's time, each for 64 of its 256 columns
          const long long until = now + (period >> 2) * (2 * u + (shares ? 0 : 1));
          while (clock64() < until) __nanosleep(64);
        }
        const long long n0 = col0 + unit * 64;
        if (row0 >= p.M || n0 >= p.N) continue;
        if (BLOCK == 16) {
          __syncwarp();   // the last unit's scales are read
          sm.gb[warp][lane] = unit ? gb[2] : gb[0];
          sm.gb[warp][lane + 32] = unit ? gb[3] : gb[1];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 64; ++i)
            acc[i >> 5][i & 31] = __float_as_uint(
                __fmul_rn(__fmul_rn(__uint_as_float(acc[i >> 5][i & 31]), ga), sm.gb[warp][i]));
        }
        store_unit(p, &tmC, tma_c, stg, acc, row0, n0, lane);
      }
    }
    if (lane == 0) bulk_wait_all();
    tc_fence_before();
  }

  chain_release();
  __syncthreads();
  if (t == 0 && sm.abort_flag) st_shared_cluster_u32(mapa_shared(smem_u32(&sm.abort_flag), rank ^ 1u), 1u);
  if (warp == NEW && rank == 0) {
    tc_fence_after();
    if (lane == 0) {
      tc_commit_pair_mc(&sm.teardown, 0x1);
      mbar_wait(&sm.teardown, 0u, nullptr, p.err, SITE_TEARDOWN);
    }
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == NEW) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, TMEM_COLS);
  }
}

template <int BLOCK>
cudaError_t launch(const GemmFp4Args& a, cudaStream_t s) {
  using C = Cfg<BLOCK>;
  auto kern = gemm_fp4_pair_kernel<BLOCK>;
  static std::mutex mu;
  static int max_clusters[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // (the occupancy query; the launch is chained)
  int clusters = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!max_clusters[dev]) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3(2 * 64, 1, 1);
      e = cudaOccupancyMaxActiveClusters(&max_clusters[dev], kern, &cfg);
      if (e != cudaSuccess) return e;
      if (max_clusters[dev] < 1) return cudaErrorInvalidConfiguration;
    }
    clusters = max_clusters[dev];
  }
  const Fp4Layout LA(a.M, a.K, BLOCK), LB(a.N, a.K, BLOCK);
  CUtensorMap ta{}, tb{}, tbp{}, tsa{}, tsb{}, tc{};
  // A's codes as rows of 1 KB (8 to a 128 x 128 tile), scales as rows of one atom, B's
  // codes by chunk (32 columns of K) and part (half or quarter) of their 128 rows
  auto parts = [](CUtensorMap* m, const uint8_t* base, const Fp4Layout& L, unsigned n) {
    const uint32_t words = 512u / n;   // 32-bit words: 128 / n rows of 16 bytes
    return make_tmap_3d(m, base, CU_TENSOR_MAP_DATA_TYPE_INT32, words, L.code_bytes() / 2048, n, 2048, words * 4, words,
                        STAGE_KT * 4, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  auto scales = [](CUtensorMap* m, const uint8_t* base, const Fp4Layout& L) {
    return make_tmap_2d(m, base + L.scale_off(), CU_TENSOR_MAP_DATA_TYPE_INT32, 128, L.scale_bytes() / 512, 512, 128,
                        STAGE_KT * C::ATOMS, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  cudaError_t e = make_tmap_2d(&ta, a.A, CU_TENSOR_MAP_DATA_TYPE_INT32, 256, LA.code_bytes() / 1024, 1024, 256,
                               STAGE_KT * 8, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e == cudaSuccess) e = parts(&tb, a.B, LB, 2);
  if (e == cudaSuccess) e = scales(&tsa, a.A, LA);
  if (e == cudaSuccess) e = scales(&tsb, a.B, LB);
  int tma_c = 0;
  if (e == cudaSuccess) e = make_c_map(a, &tc, &tma_c);
  if (e != cudaSuccess) return e;
  const int m_tiles = (int)((a.M + 255) / 256), tiles = m_tiles * (int)((a.N + 255) / 256);
  Sched sc{tiles, 1, 0, m_tiles};
  const int rest = tiles % clusters;
  if (rest > 0 && 2 * rest <= clusters) {
    sc.cut = 4 * rest <= clusters ? 4 : 2;
    sc.full = tiles - rest;
    sc.pieces = rest * sc.cut;
    if (sc.cut == 4) e = parts(&tbp, a.B, LB, 4);
  }
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(2 * (unsigned)std::min(std::max(tiles, sc.pieces), clusters), 1, 1);
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a, tma_c, sc, ta, tb, tbp, tsa, tsb, tc);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace pair
}  // namespace gfp4

cudaError_t launch_gemm_fp4_pair(const GemmFp4Args& a, int block, cudaStream_t s) {
  return block == 16 ? gfp4::pair::launch<16>(a, s) : gfp4::pair::launch<32>(a, s);
}

}  // namespace qmm
