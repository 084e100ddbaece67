// The product of two packed 4-bit matrices (fp4.cuh) on the tensor cores:
//   C[m][n] = ((sum_k a*sa * b*sb) * ga[m]) * gb[n]
// with codes a, b (e2m1), block scales sa, sb applied by the block-scaled MMA
// (tcgen05.mma kind::mxf4nvf4, fp32 accumulation in tensor memory) and the row
// scales of block 16 applied once in the epilogue (block 32 has none).
//
// One CTA per 128 x 128 tile of C: a producer warp copies each operand's codes
// and scales with bulk copies into a ring (the packed layout is the MMA's own),
// one thread moves the scales into tensor memory (tcgen05.cp) and issues the
// MMAs, four warps store the tile.
#include "common.cuh"
#include "fp4.cuh"
#include "gemm_fp4.cuh"
#include "kernels.h"

#include <algorithm>

namespace qmm {
namespace gfp4 {

constexpr int STAGE_KT = 2;                       // 128-column tiles of K per stage
constexpr int CODE_BYTES = STAGE_KT * 8192;       // per operand
constexpr int NS = 4;
constexpr int NT = 192;                           // 4 epilogue warps, MMA, producer
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t SFA_COL = 128, SFB_COL = 160;

struct Shared {
  uint64_t full[NS], empty[NS], done;
  uint32_t tmem_base;
  int abort_flag;
};

enum : unsigned { SITE_EMPTY = 0x500, SITE_FULL = 0x501, SITE_DONE = 0x502 };

template <int BLOCK>
__global__ void __launch_bounds__(NT, 1) gemm_fp4_kernel(const GemmFp4Args p) {
  constexpr int ATOMS = BLOCK == 16 ? 2 : 1;      // scale atoms per 128 columns of K
  constexpr int SF_BYTES = STAGE_KT * ATOMS * 512;
  constexpr int STAGE = 2 * CODE_BYTES + 2 * SF_BYTES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw + (sbase - raw) + NS * STAGE);
  const Fp4Layout LA(p.M, p.K, BLOCK), LB(p.N, p.K, BLOCK);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const long long mt = blockIdx.x / LB.rt, nt = blockIdx.x - mt * LB.rt;
  const int kt = (int)LA.kt, stages = (kt + STAGE_KT - 1) / STAGE_KT;
  if (t == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&sm.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  if (warp == 5) {
    if (lane == 0) {
      const uint8_t* ca = p.A + (size_t)mt * kt * 8192;
      const uint8_t* cb = p.B + (size_t)nt * kt * 8192;
      const uint8_t* fa = p.A + LA.scale_off() + (size_t)mt * kt * ATOMS * 512;
      const uint8_t* fb = p.B + LB.scale_off() + (size_t)nt * kt * ATOMS * 512;
      int s = 0;
      for (; s < stages; ++s) {
        const int slot = s % NS;
        if (s >= NS &&
            !mbar_wait(&sm.empty[slot], (uint32_t)((s / NS - 1) & 1), &sm.abort_flag, p.err, SITE_EMPTY))
          break;
        const int n = min(STAGE_KT, kt - s * STAGE_KT);
        const uint32_t dst = sbase + (uint32_t)slot * STAGE;
        mbar_arrive_expect_tx(&sm.full[slot], (uint32_t)n * 2u * (8192u + ATOMS * 512u));
        bulk_load(dst, ca + (size_t)s * CODE_BYTES, n * 8192, &sm.full[slot]);
        bulk_load(dst + CODE_BYTES, cb + (size_t)s * CODE_BYTES, n * 8192, &sm.full[slot]);
        bulk_load(dst + 2 * CODE_BYTES, fa + (size_t)s * SF_BYTES, n * ATOMS * 512, &sm.full[slot]);
        bulk_load(dst + 2 * CODE_BYTES + SF_BYTES, fb + (size_t)s * SF_BYTES, n * ATOMS * 512, &sm.full[slot]);
      }
      // no copy is left in flight when the CTA ends
      for (int j = (s > NS ? s - NS : 0); j < s; ++j)
        mbar_wait(&sm.full[j % NS], (uint32_t)((j / NS) & 1), nullptr, p.err, SITE_FULL);
    }
    __syncwarp();
  } else if (warp == 4) {
    const uint32_t on = elect_one();
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    uint32_t acc = 0u;
    for (int s = 0; s < stages; ++s) {
      const int slot = s % NS;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(&sm.full[slot], (uint32_t)((s / NS) & 1), &sm.abort_flag, p.err, SITE_FULL)))
        break;
      tc_fence_after();
      const int n = min(STAGE_KT, kt - s * STAGE_KT);
      const uint32_t a = (sbase + (uint32_t)slot * STAGE) >> 4, b = a + (CODE_BYTES >> 4);
      const uint32_t fa = b + (CODE_BYTES >> 4), fb = fa + (SF_BYTES >> 4);
      for (int i = 0; i < n * ATOMS; ++i) {
        cp_scales(tb + SFA_COL + i * 4, fa + i * 32, on);
        cp_scales(tb + SFB_COL + i * 4, fb + i * 32, on);
      }
      for (int j = 0; j < 2 * n; ++j) {   // 64 columns of K each
        const uint32_t col = BLOCK == 16 ? j * 4 : (j >> 1) * 4;
        mma_fp4<BLOCK>(tb, a + j * 256 + kDescLo, b + j * 256 + kDescLo,
                       idesc_fp4(128, 128, BLOCK == 32, BLOCK == 32 ? (j & 1) * 2 : 0), tb + SFA_COL + col,
                       tb + SFB_COL + col, acc, on);
        acc = 1u;
      }
      commit_on(&sm.empty[slot], on);
    }
    commit_on(&sm.done, on);   // also after a wait that ran out: every MMA issued so far
    __syncwarp();
  } else {
    const long long row = mt * 128 + warp * 32 + lane;
    const bool ok = mbar_wait(&sm.done, 0u, nullptr, p.err, SITE_DONE, 4 * kWaitLimitNs);
    tc_fence_after();
    const float ga = (BLOCK == 16 && row < p.M) ? reinterpret_cast<const float*>(p.A + LA.row_off())[row] : 1.f;
    for (int g = 0; g < 4; ++g) {
      uint32_t acc[32];
      tmem_ld32(tbase + ((uint32_t)(warp * 32) << 16) + g * 32, acc);
      for (int i = 0; i < 32; ++i) {
        const long long n = nt * 128 + g * 32 + i;
        if (!ok || sm.abort_flag || row >= p.M || n >= p.N) continue;
        float v = __uint_as_float(acc[i]);
        if (BLOCK == 16)
          v = __fmul_rn(__fmul_rn(v, ga), __ldg(reinterpret_cast<const float*>(p.B + LB.row_off()) + n));
        if (p.c_f32) static_cast<float*>(p.C)[row * p.N + n] = v;
        else static_cast<__nv_bfloat16*>(p.C)[row * p.N + n] = __float2bfloat16_rn(v);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

template <int BLOCK>
cudaError_t launch(const GemmFp4Args& a, cudaStream_t s) {
  constexpr int ATOMS = BLOCK == 16 ? 2 : 1;
  const size_t smem = NS * (2 * CODE_BYTES + 2 * STAGE_KT * ATOMS * 512) + sizeof(Shared) + 1024;
  cudaError_t e = cudaFuncSetAttribute(gemm_fp4_kernel<BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const Fp4Layout LA(a.M, a.K, BLOCK), LB(a.N, a.K, BLOCK);
  gemm_fp4_kernel<BLOCK><<<(unsigned)(LA.rt * LB.rt), NT, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace gfp4

cudaError_t launch_gemm_fp4(const GemmFp4Args& a, int block, cudaStream_t s, const char** kernel_name) {
  if (a.M > 256) {
    *kernel_name = "gemm_fp4_pair";
    return launch_gemm_fp4_pair(a, block, s);
  }
  *kernel_name = "gemm_fp4";
  return block == 16 ? gfp4::launch<16>(a, s) : gfp4::launch<32>(a, s);
}

}  // namespace qmm
