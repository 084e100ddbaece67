// Block-scaled 4-bit MMA pieces shared by the products of packed 4-bit matrices.
#pragma once

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "tma.h"

#include <climits>

namespace qmm {
namespace gfp4 {

// Instruction descriptor of the block-scaled 4-bit MMA: [4,6) B scale id,
// [7,10) A format (1 = e2m1), [10,13) B format, [17,23) N >> 3, 23 scale type
// (0 = ue4m3, 1 = ue8m0), [24,29) M >> 4, [29,31) A scale id; 31: K = 64. The
// scale id is the byte of a 32-bit scale word that the instruction starts at.
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, bool e8m0, int sf_id) {
  return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) |
         ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf_id << 29);
}

// Shared-memory descriptor without swizzle (K-major): [0,14) address / 16,
// [16,30) bytes between core matrices along K / 16, [32,46) bytes between 8-row
// groups / 16, 46 version. Here always 2 KB between core matrices along K and 128
// bytes between 8-row groups (the packed layout), so the low word is
// address / 16 + kDescLo. (The scale copies use the 8-row groups alone.)
// A shared address as a descriptor holds it. In a cluster the addresses of CTAs
// past the first have higher bits set, which would land in the next field.
__device__ __forceinline__ uint32_t desc_addr(uint32_t saddr) { return (saddr >> 4) & 0x3FFFu; }
constexpr uint32_t kDescLo = (2048u >> 4) << 16;
constexpr uint32_t kDescHi = (128u >> 4) | (1u << 14);

// The MMA warp runs converged and one lane issues (`on` is that lane's flag):
// addresses and descriptors then stay in uniform registers, where the
// instructions take them from. Issued from inside a one-lane branch, every
// operand is moved there first, and that thread's own instructions, not the
// tensor core, set the rate.
//
// D[tmem] (+)= (A scaled) x (B scaled): 16 (4 scales a K step) or 32 (2) elements to a scale.
#define QMM_FP4_MMA(GROUP, VEC)                                                                                    \
  asm volatile(                                                                                                    \
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"                                                               \
      "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 e, %7, 0;\n\t"                                                         \
      "mov.b64 a, {%1, %8};\n\tmov.b64 b, {%2, %8};\n\t"                                                           \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                             \
      " [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                                             \
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(on), "r"(kDescHi)                        \
      : "memory")
template <int BLOCK>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t acc, uint32_t on) {
  if (BLOCK == 16) QMM_FP4_MMA("1", "4X");
  else QMM_FP4_MMA("1", "2X");
}
template <int BLOCK>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t acc, uint32_t on) {
  if (BLOCK == 16) QMM_FP4_MMA("2", "4X");
  else QMM_FP4_MMA("2", "2X");
}

// One atom of scales (512 bytes at 16 * addr16) into four tensor-memory columns,
// repeated in the four 32-lane quarters. Executes in order with the MMAs of the
// same thread.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint32_t addr16, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 a;\n\tsetp.ne.b32 e, %2, 0;\n\tmov.b64 a, {%1, %3};\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], a;\n\t}" ::"r"(taddr),
      "r"(addr16), "r"(on), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint32_t addr16, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 a;\n\tsetp.ne.b32 e, %2, 0;\n\tmov.b64 a, {%1, %3};\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], a;\n\t}" ::"r"(taddr),
      "r"(addr16), "r"(on), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit_on(uint64_t* bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_pair_on(uint64_t* bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3), "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(on));
  return on;
}

__device__ __forceinline__ uint32_t pack_bf16(uint32_t a, uint32_t b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<uint32_t*>(&v);
}

// A warp's 32 rows x 64 columns of C (one row a lane) to memory through its
// staging buffer: 32 rows x 128 bytes (64 bf16 or twice 32 f32 columns), 16-byte
// chunk j of row r at chunk j ^ (r & 7) (the 128-byte swizzle, conflict-free).
// tma: one lane stores the box (what lies outside C is not written); otherwise
// the warp writes each staged row element by element.
__device__ __forceinline__ void store_box(const GemmFp4Args& p, const CUtensorMap* tmC, int tma, uint32_t stg,
                                          const uint32_t (&w)[32], long long row0, long long n0, int lane) {
  if (tma) {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_shared_v4(stg + (uint32_t)lane * 128u + (uint32_t)((j ^ (lane & 7)) * 16), w[4 * j], w[4 * j + 1], w[4 * j + 2],
                 w[4 * j + 3]);
  if (tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmC), "r"(stg),
                   "r"((int)n0), "r"((int)row0)
                   : "memory");
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  const int rows = (int)min(32ll, p.M - row0);
  const int n = (int)min((long long)INT_MAX, p.N - n0);   // columns from n0 on
  uint8_t* c = static_cast<uint8_t*>(p.C) + (row0 * p.N + n0) * (p.c_f32 ? 4 : 2);
  const long long pitch = p.N * (p.c_f32 ? 4 : 2);
  for (int r0 = 0; r0 < rows; r0 += 8) {   // eight rows at a time: each waits for its words
    uint32_t v[8];   // this lane's 4 bytes of the rows
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a =
          stg + (uint32_t)(r0 + i) * 128u + (uint32_t)((((lane >> 2) ^ ((r0 + i) & 7)) << 4) + (lane & 3) * 4);
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[i]) : "r"(a));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i >= rows) break;
      if (p.c_f32) {
        if (lane < n) reinterpret_cast<uint32_t*>(c)[lane] = v[i];
      } else {   // (shifting pairs to 4-byte boundaries through shuffles was slower)
        uint16_t* h = reinterpret_cast<uint16_t*>(c) + 2 * lane;
        if (2 * lane < n) h[0] = (uint16_t)v[i];
        if (2 * lane + 1 < n) h[1] = (uint16_t)(v[i] >> 16);
      }
      c += pitch;
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void store_unit(const GemmFp4Args& p, const CUtensorMap* tmC, int tma, uint32_t stg,
                                           const uint32_t (&acc)[2][32], long long row0, long long n0, int lane) {
  if (p.c_f32) {
    store_box(p, tmC, tma, stg, acc[0], row0, n0, lane);
    if (n0 + 32 < p.N) store_box(p, tmC, tma, stg, acc[1], row0, n0 + 32, lane);
  } else {
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = pack_bf16(acc[i >> 4][(2 * i) & 31], acc[i >> 4][(2 * i + 1) & 31]);
    store_box(p, tmC, tma, stg, w, row0, n0, lane);
  }
}

// C as a matrix of 128-byte wide boxes of 32 rows, where its pitch allows.
inline cudaError_t make_c_map(const GemmFp4Args& a, CUtensorMap* tc, int* tma) {
  const int es = a.c_f32 ? 4 : 2;
  *tma = (reinterpret_cast<uintptr_t>(a.C) % 16) == 0 && (a.N * es) % 16 == 0;
  if (!*tma) return cudaSuccess;
  return make_tmap_2d(tc, a.C, a.c_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.N * es, 128 / es, 32, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace gfp4
}  // namespace qmm
