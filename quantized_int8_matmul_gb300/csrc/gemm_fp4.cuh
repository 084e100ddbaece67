// Block-scaled 4-bit MMA pieces shared by the products of packed 4-bit matrices.
#pragma once

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "tma.h"

namespace qmm {
namespace gfp4 {

// Shared-memory descriptor without swizzle (K-major): lbo bytes between core
// matrices (8 rows x 16 bytes) along K, sbo bytes between 8-row groups.
__device__ __forceinline__ uint64_t sdesc_none(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// Instruction descriptor of the block-scaled 4-bit MMA: [4,6) B scale id,
// [7,10) A format (1 = e2m1), [10,13) B format, [17,23) N >> 3, 23 scale type
// (0 = ue4m3, 1 = ue8m0), [24,29) M >> 4, [29,31) A scale id; 31: K = 64. The
// scale id is the byte of a 32-bit scale word that the instruction starts at.
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, bool e8m0, int sf_id) {
  return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) |
         ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf_id << 29);
}

// D[tmem] (+)= (A scaled) x (B scaled): 16 (4 scales a K step) or 32 (2) elements to a scale.
template <int BLOCK>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t acc) {
  if (BLOCK == 16)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
template <int BLOCK>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t acc) {
  if (BLOCK == 16)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// One atom of scales (512 bytes) into four tensor-memory columns, repeated in
// the four 32-lane quarters. Executes in order with the MMAs of the same thread.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
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
  for (int r = 0; r < rows; ++r) {
    uint32_t v;   // this lane's 4 bytes of the row
    const uint32_t a = stg + (uint32_t)r * 128u + (uint32_t)((((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    const long long row = row0 + r;
    if (p.c_f32) {
      const long long n = n0 + lane;
      if (n < p.N) static_cast<uint32_t*>(p.C)[row * p.N + n] = v;
    } else {
      const long long n = n0 + 2 * lane;
      uint16_t* c = static_cast<uint16_t*>(p.C) + row * p.N + n;
      if (n < p.N) c[0] = (uint16_t)v;
      if (n + 1 < p.N) c[1] = (uint16_t)(v >> 16);
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
