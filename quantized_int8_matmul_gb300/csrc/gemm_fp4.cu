// The product of two packed 4-bit matrices (fp4.cuh) for up to 64 rows of A:
//   C[m][n] = ((sum_k a*sa * b*sb) * ga[m]) * gb[n]
// (the MMA and its operands as in gemm_fp4_pair.cu). A few rows of activations
// against a weight read 0.53 or 0.56 bytes an element of the weight from HBM and
// do little else, so the roles are swapped: 128 rows of B (columns of C) are the
// MMA's M side, and all rows of A, rounded up to 16, its N side. Every byte of
// the weight is read by exactly one CTA.
//
// A cluster of S CTAs shares 128 columns of C, each taking a run of K: S is the
// largest (up to 8) that keeps all CTAs resident at once, two an SM. Each CTA
// (192 threads): warp 5 copies the weight's codes and scales (256 columns of K a
// stage, one contiguous run each) and the rows' chunks into a ring with bulk
// copies; warp 4 moves the scales to tensor memory and issues the MMAs; warps
// 0-3 put the fp32 partial sums in shared memory, and after a cluster barrier
// each CTA adds up its share of the rows over the cluster in rank order (so the
// result does not depend on timing), scales and stores them.
// 1 x 28672 x 8192: block 16 21.7 us, block 32 20.1 (6.1 and 6.2 TB/s of weight and
// scales, 91 and 93 % of a copy's rate); 64 x 28672 x 8192 25.6 and 23.1. 1 x 4096 x
// 4096 5.5 and 5.1 us, of which the weight's bytes are 1.4: the launch, the first
// bytes' way and the join over the cluster (0.9 us) are the rest.
// Every wait is bounded (common.cuh).
#include "chain.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "gemm_fp4.cuh"
#include "kernels.h"

#include <algorithm>
#include <mutex>

namespace qmm {
namespace gfp4 {
namespace rows {

constexpr int STAGE_KT = 2;                       // 128-column tiles of K per stage
constexpr int CODE_BYTES = STAGE_KT * 8192;       // the weight's codes per stage
constexpr int NS_MAX = 8;
constexpr int NT = 192;                           // 4 epilogue warps, MMA, producer

struct Shared {
  uint64_t full[NS_MAX], empty[NS_MAX], done;
  uint32_t tmem_base;
  int abort_flag;
};

enum : unsigned { SITE_EMPTY = 0x500, SITE_FULL = 0x501, SITE_DONE = 0x502 };

// What the host chose for a problem.
struct Plan {
  int mp;        // rows of A rounded up to 16
  int ns;        // ring stages
  int split;     // CTAs of a cluster (each a run of K)
  int stage;     // bytes of a stage
  int tmem;      // tensor memory columns
  size_t smem;
};

template <int BLOCK>
struct Cfg {
  static constexpr int ATOMS = BLOCK == 16 ? 2 : 1;
  static constexpr int SF_BYTES = STAGE_KT * ATOMS * 512;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <int BLOCK>
__global__ void __launch_bounds__(NT, 2) gemm_fp4_rows_kernel(const GemmFp4Args p, const Plan pl) {
  constexpr int ATOMS = Cfg<BLOCK>::ATOMS, SF_BYTES = Cfg<BLOCK>::SF_BYTES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 127u) & ~127u;
  uint8_t* sptr = smem_raw + (sbase - raw);
  Shared& sm = *reinterpret_cast<Shared*>(sptr + (size_t)pl.ns * pl.stage);
  const Fp4Layout LA(p.M, p.K, BLOCK), LB(p.N, p.K, BLOCK);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = pl.split > 1 ? (int)cluster_ctarank() : 0;
  const long long nt = blockIdx.x / pl.split;
  const int kt = (int)LA.kt, stages_all = (kt + STAGE_KT - 1) / STAGE_KT;
  const int s0 = (int)((long long)stages_all * rank / pl.split);
  const int s1 = (int)((long long)stages_all * (rank + 1) / pl.split);
  const int mp = pl.mp;
  const uint32_t sf_col = (uint32_t)(mp + 31) & ~31u;
  if (t == 0) {
    for (int i = 0; i < pl.ns; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&sm.tmem_base, (uint32_t)pl.tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  chain_wait();   // what is above ran under the call before

  if (warp == 5) {
    // ---------------- producer ----------------
    if (lane == 0) {
      const uint8_t* wc = p.B + (size_t)nt * kt * 8192;
      const uint8_t* wf = p.B + LB.scale_off() + (size_t)nt * kt * ATOMS * 512;
      const uint8_t* xf = p.A + LA.scale_off();
      int slot = 0;
      uint32_t phase = 1u;   // a fresh ring slot is empty
      int s = s0;
      for (; s < s1; ++s) {
        if (s - s0 >= pl.ns && !mbar_wait(&sm.empty[slot], phase, &sm.abort_flag, p.err, SITE_EMPTY)) break;
        const int n = min(STAGE_KT, kt - s * STAGE_KT);
        const uint32_t dst = sbase + (uint32_t)(slot * pl.stage);
        uint64_t* bar = &sm.full[slot];
        mbar_arrive_expect_tx(bar, (uint32_t)n * (8192u + (uint32_t)mp * 64u + 2u * ATOMS * 512u));
        bulk_load(dst, wc + (size_t)s * CODE_BYTES, n * 8192, bar);
        bulk_load(dst + CODE_BYTES, wf + (size_t)s * SF_BYTES, n * ATOMS * 512, bar);
        bulk_load(dst + CODE_BYTES + SF_BYTES, xf + (size_t)s * SF_BYTES, n * ATOMS * 512, bar);
        for (int c = 0; c < 4 * n; ++c)
          bulk_load(dst + CODE_BYTES + 2 * SF_BYTES + (uint32_t)(c * mp * 16),
                    p.A + (size_t)s * CODE_BYTES + c * 2048, (uint32_t)mp * 16u, bar);
        if (++slot == pl.ns) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // no copy is left in flight when the CTA ends
      for (int j = (s - s0 > pl.ns ? s - pl.ns : s0); j < s; ++j)
        mbar_wait(&sm.full[(j - s0) % pl.ns], (uint32_t)(((j - s0) / pl.ns) & 1), nullptr, p.err, SITE_FULL);
    }
    __syncwarp();
  } else if (warp == 4) {
    // ---------------- MMA issuer (the warp converged) ----------------
    const uint32_t on = elect_one();
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t id0 = idesc_fp4(128, 0, BLOCK == 32, 0) | ((uint32_t)(mp >> 3) << 17);
    const uint32_t id1 = idesc_fp4(128, 0, BLOCK == 32, 2) | ((uint32_t)(mp >> 3) << 17);
    const uint32_t s16 = desc_addr(sbase);
    const uint32_t x_lbo = (uint32_t)mp << 16;      // bytes between A's chunks / 16
    const uint32_t sa0 = tb + sf_col, sb0 = sa0 + STAGE_KT * ATOMS * 4;
    int slot = 0;
    uint32_t phase = 0u, acc = 0u;
    for (int s = s0; s < s1; ++s) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[slot], phase, &sm.abort_flag, p.err, SITE_FULL))) break;
      tc_fence_after();
      const uint32_t w = s16 + (uint32_t)(slot * pl.stage >> 4), wf = w + (CODE_BYTES >> 4);
      const uint32_t xf = wf + (SF_BYTES >> 4), x = xf + (SF_BYTES >> 4);
      const int n = min(STAGE_KT, kt - s * STAGE_KT);
#pragma unroll
      for (int k = 0; k < STAGE_KT; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int i = 0; i < ATOMS; ++i) {
          const int q = k * ATOMS + i;
          cp_scales(sa0 + q * 4, wf + q * 32, on);
          cp_scales(sb0 + q * 4, xf + q * 32, on);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // 64 columns of K each: two chunks
          const int q = BLOCK == 16 ? k * 2 + j : k;
          mma_fp4<BLOCK>(tb, w + (uint32_t)(k * 512 + j * 256) + kDescLo, x + (uint32_t)((k * 4 + j * 2) * mp) + x_lbo,
                         (BLOCK == 32 && j) ? id1 : id0, sa0 + q * 4, sb0 + q * 4, acc, on);
          acc = 1u;
        }
      }
      commit_on(&sm.empty[slot], on);
      if (++slot == pl.ns) {
        slot = 0;
        phase ^= 1u;
      }
    }
    commit_on(&sm.done, on);   // also after a wait that ran out: every MMA issued so far
    __syncwarp();
  }
  // ---------------- partial sums to shared memory: part[m][128] ----------------
  const bool ok = mbar_wait(&sm.done, 0u, nullptr, p.err, SITE_DONE, 4 * kWaitLimitNs);
  chain_release();
  tc_fence_after();
  // the ring is free: every copy has landed (the MMAs that completed waited for
  // them all, or the producer did before this barrier)
  __syncthreads();
  float* part = reinterpret_cast<float*>(sptr);
  if (warp < 4 && ok) {
    for (int g = 0; g < mp; g += 16) {
      uint32_t acc[16];
      tmem_ld16(tbase + ((uint32_t)(warp * 32) << 16) + g, acc);
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(g + i) * 128 + warp * 32 + lane] = __uint_as_float(acc[i]);
    }
    tc_fence_before();
  }
  if (pl.split > 1) cluster_sync_all();
  else __syncthreads();
  // ---------------- this CTA's rows: sum over the cluster, scale, store ----------------
  const long long n0 = nt * 128 + lane * 4;
  float gb[4] = {1.f, 1.f, 1.f, 1.f};
  if (BLOCK == 16) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n0 + e < p.N) gb[e] = __ldg(reinterpret_cast<const float*>(p.B + LB.row_off()) + n0 + e);
  }
  const bool v4 = (p.N & 3) == 0 && (reinterpret_cast<uintptr_t>(p.C) & 15) == 0;
  if (ok && !sm.abort_flag) {
    for (int m = rank + warp * pl.split; m < p.M; m += (NT / 32) * pl.split) {
      const uint32_t local = sbase + (uint32_t)(m * 512 + lane * 16);
      float4 v = pl.split > 1 ? ld_cluster_f4(mapa_shared(local, 0))
                              : *reinterpret_cast<const float4*>(part + m * 128 + lane * 4);
      for (int r = 1; r < pl.split; ++r) {
        const float4 o = ld_cluster_f4(mapa_shared(local, (uint32_t)r));
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
      if (BLOCK == 16) {
        const float ga = __ldg(reinterpret_cast<const float*>(p.A + LA.row_off()) + m);
        v.x = __fmul_rn(__fmul_rn(v.x, ga), gb[0]);
        v.y = __fmul_rn(__fmul_rn(v.y, ga), gb[1]);
        v.z = __fmul_rn(__fmul_rn(v.z, ga), gb[2]);
        v.w = __fmul_rn(__fmul_rn(v.w, ga), gb[3]);
      }
      if (n0 >= p.N) continue;
      if (p.c_f32) {
        float* c = static_cast<float*>(p.C) + (long long)m * p.N + n0;
        if (v4) {
          *reinterpret_cast<float4*>(c) = v;
        } else {
          const float e[4] = {v.x, v.y, v.z, v.w};
          for (int i = 0; i < 4 && n0 + i < p.N; ++i) c[i] = e[i];
        }
      } else {
        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.C) + (long long)m * p.N + n0;
        const uint32_t lo = pack_bf16(__float_as_uint(v.x), __float_as_uint(v.y));
        const uint32_t hi = pack_bf16(__float_as_uint(v.z), __float_as_uint(v.w));
        if (v4) {
          *reinterpret_cast<uint2*>(c) = make_uint2(lo, hi);
        } else {
          const uint32_t w[2] = {lo, hi};
          for (int i = 0; i < 4 && n0 + i < p.N; ++i)
            reinterpret_cast<uint16_t*>(c)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
      }
    }
  }
  if (pl.split > 1) cluster_sync_all();   // the others have read this CTA's sums
  else __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tbase, (uint32_t)pl.tmem);
  }
}

// Ring and split for a problem: two CTAs an SM (their rings and tensor memory),
// and the largest split that keeps every CTA resident at once, each with two
// stages at least. 1 x 28672 x 8192 (224 column tiles): 21.7 us with a split of
// 1, 29.8 with 2 (448 CTAs, a second wave); 1 x 4096 x 4096 (32 tiles): 12.0
// with 1, 6.6 with 4, 6.9 with 8.
template <int BLOCK>
Plan make_plan(const GemmFp4Args& a) {
  Plan pl;
  const Fp4Layout LB(a.N, a.K, BLOCK);
  pl.mp = (int)((a.M + 15) / 16 * 16);
  const int sf = Cfg<BLOCK>::SF_BYTES;
  pl.stage = CODE_BYTES + 2 * sf + pl.mp * 16 * 4 * STAGE_KT;
  pl.ns = std::min(NS_MAX, 110 * 1024 / pl.stage);   // at least 3; the partial sums (mp * 512) fit in one stage or two
  const int cols = ((pl.mp + 31) & ~31) + 2 * STAGE_KT * Cfg<BLOCK>::ATOMS * 4;
  pl.tmem = cols <= 64 ? 64 : 128;
  const long long stages = (LB.kt + STAGE_KT - 1) / STAGE_KT;
  pl.split = (int)std::max<long long>(1, std::min({8ll, 2ll * num_sms() / LB.rt, stages / 2}));
  pl.smem = (size_t)pl.ns * pl.stage + sizeof(Shared) + 128;
  return pl;
}

template <int BLOCK>
cudaError_t launch(const GemmFp4Args& a, cudaStream_t s) {
  auto kern = gemm_fp4_rows_kernel<BLOCK>;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
      if (e != cudaSuccess) return e;
      ready[dev] = true;
    }
  }
  const Plan pl = make_plan<BLOCK>(a);
  const Fp4Layout LB(a.N, a.K, BLOCK);
  return launch_chained(kern, (unsigned)(LB.rt * pl.split), NT, pl.smem, (unsigned)pl.split, s, a, pl);
}

}  // namespace rows
}  // namespace gfp4

cudaError_t launch_gemm_fp4(const GemmFp4Args& a, int block, cudaStream_t s, const char** kernel_name) {
  // Above 64 rows the pair kernel's 256 x 256 tiles win although they may be
  // mostly padding: 128 x 11008 x 4096 takes 11.1 us there and 14.3 here, 64 rows
  // 10.5 and 10.2, 64 x 28672 x 8192 30.0 and 25.6.
  if (a.M > 64) {
    *kernel_name = "gemm_fp4_pair";
    return launch_gemm_fp4_pair(a, block, s);
  }
  *kernel_name = "gemm_fp4_rows";
  return block == 16 ? gfp4::rows::launch<16>(a, s) : gfp4::rows::launch<32>(a, s);
}

}  // namespace qmm
