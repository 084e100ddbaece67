// Quantisation of a float matrix to 4-bit floats (e2m1) with block scales,
// along its rows, its columns, or both from one read; and reading back.
//
// block 32 (a power of two per 32 elements, as in the OCP Microscaling Formats
// specification, MXFP4): with b the block's largest magnitude, the scale is
// 2^(floor(log2 b) - 2), at least 2^-127, and the codes are x / scale rounded
// to the nearest e2m1 (ties to even, beyond 6 to 6). Every step but the last
// rounding is exact.
// block 16 (an e4m3 scale per 16 elements under a float32 scale per row):
// g = rowmax / 2688 (6 * 448; 1 where that is below 2^-100: such a row is
// stored as zeros), u = 1 / g, s = e4m3(b * u / 6), codes = e2m1(x * (u / s)).
// The row scale is per row and not per tensor so that one pass over a row
// settles it; the product applies it in its epilogue.
// A block (32) or row (16) that holds a NaN or an infinity gets a NaN scale.
//
// Bound by HBM: x is read once, 0.53 or 0.56 bytes an element are written.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"

#include <algorithm>
#include <cuda_fp8.h>

namespace qmm {
namespace fp4 {

constexpr unsigned kInfBits = 0x7f800000u;
constexpr float kR2688 = 1.0f / 2688.0f;
constexpr float kR6 = 1.0f / 6.0f;

// Eight floats to eight e2m1 codes, element 0 in the lowest 4 bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ float e4m3_to_f(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}
__device__ __forceinline__ float e8m0_to_f(uint8_t b) {
  return __uint_as_float(b == 255 ? 0x7fffffffu : b == 0 ? 0x00400000u : (uint32_t)b << 23);
}

// The row's float32 scale from the bits of its largest magnitude.
__device__ __forceinline__ float row_scale(unsigned max_bits) {
  if (max_bits >= kInfBits) return __uint_as_float(0x7fffffffu);
  const float g = __fmul_rn(__uint_as_float(max_bits), kR2688);
  return g < 0x1p-100f ? 1.f : g;
}

// One block's scale byte and the multiplier of its elements, from the bits of
// its largest magnitude. BLOCK 16: u = 1 / row scale (NaN: zeros). zero: the
// codes are zeros whatever the elements are.
template <int BLOCK>
__device__ __forceinline__ uint8_t block_scale(unsigned max_bits, float u, float& mul, bool& zero) {
  if (BLOCK == 32) {
    zero = max_bits >= kInfBits;
    const int byte = max((int)(max_bits >> 23) - 2, 0);
    mul = __uint_as_float((uint32_t)(254 - byte) << 23);
    return zero ? 255 : (uint8_t)byte;
  }
  const float t = __fmul_rn(__fmul_rn(__uint_as_float(max_bits), u), kR6);
  zero = !(t > 0.f) || !(u > 0.f);
  if (zero) return 0;
  const uint8_t b = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  zero = b == 0;
  mul = zero ? 0.f : __fdiv_rn(u, e4m3_to_f(b));
  return b;
}

template <typename T>
__device__ __forceinline__ float ld1(const T* p);
template <>
__device__ __forceinline__ float ld1<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float ld1<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Elements [k, k + 8) of a row of n (k a multiple of 8; past the end: 0).
template <typename T>
__device__ __forceinline__ void load8(const T* row, long long k, long long n, bool vec, float (&v)[8]) {
  if (vec && k + 8 <= n) {
    if (sizeof(T) == 2) {
      const uint4 r = *reinterpret_cast<const uint4*>(row + k);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(row + k);
      const float4 b = *(reinterpret_cast<const float4*>(row + k) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < n ? ld1(row + k + e) : 0.f;
  }
}

__device__ __forceinline__ unsigned max8(const float (&v)[8]) {
  unsigned m = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  return m;
}

// The maximum over the lanes that share a block: 4 lanes of 8 elements for 32,
// 2 for 16.
template <int BLOCK>
__device__ __forceinline__ unsigned block_max(unsigned m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (BLOCK == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return m;
}

// ---------------------------------------------------------------------------
// Along the rows. A CTA takes eight rows of a tile, {2c, 2c + 1} + {0, 32, 64,
// 96}, a warp 32 columns of them at a time: lane l holds 8 columns of row l / 4.
// Rows chosen so make every 32-byte sector of codes (two neighbouring rows'
// 16 bytes) and of scales (two rows' 16-byte lines of an atom, whose 4-byte
// parts are rows 32 apart) the work of one CTA.
// ---------------------------------------------------------------------------
template <typename T, int BLOCK>
__global__ void quantize_rows_kernel(const Fp4QuantArgs p) {
  constexpr int SPC = 32 / BLOCK;   // scales per 32-column chunk
  __shared__ unsigned rowmax[8];
  const Fp4Layout L(p.rows, p.cols, BLOCK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const long long tile = blockIdx.x >> 4;
  const int rin = 2 * (blockIdx.x & 15) + ((lane >> 2) & 1) + 32 * (lane >> 3);
  const long long row = tile * 128 + rin;
  if (tile * 128 + 2 * (blockIdx.x & 15) >= p.rows) return;
  const bool rv = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + (rv ? row : 0) * p.ld;
  const long long n = rv ? p.cols : 0;
  const bool vec = p.vec;
  const int chunks = (int)(L.kt * 4);
  float u = 1.f;
  if (BLOCK == 16) {
    if (threadIdx.x < 8) rowmax[threadIdx.x] = 0u;
    __syncthreads();
    unsigned m = 0u;
    for (int c = warp; c < chunks; c += nw) {
      float v[8];
      load8(x, (long long)c * 32 + (lane & 3) * 8, n, vec, v);
      m = max(m, max8(v));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if ((lane & 3) == 0) atomicMax(&rowmax[lane >> 2], m);
    __syncthreads();
    const float g = row_scale(rowmax[lane >> 2]);
    u = __fdiv_rn(1.f, g);
    if (warp == 0 && (lane & 3) == 0 && rv) reinterpret_cast<float*>(p.out + L.row_off())[row] = g;
  }
  uint8_t* codes = p.out + (size_t)tile * L.kt * 8192 + rin * 16 + (lane & 3) * 4;
  uint8_t* sf = p.out + L.scale_off() + (size_t)tile * L.kt * 512 * L.atoms() + (rin & 31) * 16 + (rin >> 5) * 4;
  for (int c = warp; c < chunks; c += nw) {
    float v[8];
    load8(x, (long long)c * 32 + (lane & 3) * 8, n, vec, v);
    float mul = 0.f;
    bool zero;
    const uint8_t s = block_scale<BLOCK>(block_max<BLOCK>(max8(v)), u, mul, zero);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], mul);
    const uint32_t code = zero ? 0u : e2m1x8(v);
    if (rv) {
      *reinterpret_cast<uint32_t*>(codes + (size_t)c * 2048) = code;
      const int k = c * SPC + (BLOCK == 16 ? (lane & 3) >> 1 : 0);
      if ((lane & (BLOCK == 16 ? 1 : 3)) == 0) sf[(size_t)(k >> 2) * 512 + (k & 3)] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// Along the columns, or both ways: x is [rows][cols] in memory; the packed
// matrix along the columns is its transpose [cols][rows]. A CTA takes a tile of
// 128 x 128 of x through shared memory.
// ---------------------------------------------------------------------------
// Largest magnitudes of the columns (and the rows) into the packed buffers' max words.
template <typename T>
__global__ void absmax_kernel(const Fp4QuantArgs p, unsigned* colmax, unsigned* rowmax) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kt = (int)((p.cols + 127) / 128), ty = blockIdx.x / kt, tx = blockIdx.x - ty * kt;
  const long long c0 = (long long)tx * 128, r0 = (long long)ty * 128;
  unsigned cm[4] = {0u, 0u, 0u, 0u};
  for (int i = warp; i < 128; i += 8) {
    const long long r = r0 + i;
    if (r >= p.rows) break;
    unsigned rm = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long c = c0 + j * 32 + lane;
      const unsigned b =
          c < p.cols ? __float_as_uint(ld1(static_cast<const T*>(p.x) + r * p.ld + c)) & 0x7fffffffu : 0u;
      cm[j] = max(cm[j], b);
      rm = max(rm, b);
    }
    if (rowmax) {
      rm = __reduce_max_sync(0xffffffffu, rm);
      if (lane == 0) atomicMax(rowmax + r, rm);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long c = c0 + j * 32 + lane;
    if (c < p.cols) atomicMax(colmax + c, cm[j]);
  }
}

template <typename T, int BLOCK, bool ROWS>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const Fp4QuantArgs p) {
  constexpr int SPC = 32 / BLOCK;
  extern __shared__ __align__(16) uint8_t smem[];
  T* tile = reinterpret_cast<T*>(smem);   // [128][128]
  __shared__ __align__(16) uint8_t sfs[1024];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const Fp4Layout Lr(p.rows, p.cols, BLOCK), Lc(p.cols, p.rows, BLOCK);
  const int ty = blockIdx.x / (int)Lr.kt, tx = blockIdx.x - ty * (int)Lr.kt;
  const long long c0 = (long long)tx * 128, r0 = (long long)ty * 128;
  const size_t ti = blockIdx.x;                       // this tile in the packed rows
  const size_t tc = (size_t)tx * Lc.kt + ty;          // and in the packed columns
  // rows of x: quantised as they are loaded
#pragma unroll 2
  for (int it = 0; it < 8; ++it) {
    const int item = it * 8 + warp, ch = item & 3, grp = item >> 2;
    const int rin = 2 * grp + ((lane >> 2) & 1) + 32 * (lane >> 3);
    const long long row = r0 + rin;
    const bool rv = row < p.rows;
    const int k = ch * 32 + (lane & 3) * 8;
    float v[8];
    load8(static_cast<const T*>(p.x) + (rv ? row : 0) * p.ld, c0 + k, rv ? p.cols : 0, p.vec, v);
    T* d = tile + rin * 128 + k;
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = (T)v[e];
    if (ROWS) {
      float u = 1.f, mul = 0.f;
      if (BLOCK == 16) {
        const float g = row_scale(rv ? reinterpret_cast<const unsigned*>(p.out_rows + Lr.max_off())[row] : 0u);
        u = __fdiv_rn(1.f, g);
        if (c0 == 0 && ch == 0 && (lane & 3) == 0 && rv) reinterpret_cast<float*>(p.out_rows + Lr.row_off())[row] = g;
      }
      bool zero;
      const uint8_t s = block_scale<BLOCK>(block_max<BLOCK>(max8(v)), u, mul, zero);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], mul);
      const uint32_t code = zero ? 0u : e2m1x8(v);
      *reinterpret_cast<uint32_t*>(p.out_rows + ti * 8192 + ch * 2048 + rin * 16 + (lane & 3) * 4) = code;
      const int ks = ch * SPC + (BLOCK == 16 ? (lane & 3) >> 1 : 0);
      if ((lane & (BLOCK == 16 ? 1 : 3)) == 0)
        sfs[(ks >> 2) * 512 + (rin & 31) * 16 + (rin >> 5) * 4 + (ks & 3)] = s;
    }
  }
  __syncthreads();
  if (ROWS) {
    if (t < 32 * Lr.atoms())
      reinterpret_cast<uint4*>(p.out_rows + Lr.scale_off() + ti * 512 * Lr.atoms())[t] =
          reinterpret_cast<const uint4*>(sfs)[t];
    __syncthreads();
  }
  // columns: one column and 32 rows at a time
  for (int item = t; item < 512; item += 256) {
    const int c = item & 127, ch = item >> 7;
    const bool cv = c0 + c < p.cols;
    float u = 1.f;
    if (BLOCK == 16) {
      const float g = row_scale(cv ? reinterpret_cast<const unsigned*>(p.out + Lc.max_off())[c0 + c] : 0u);
      u = __fdiv_rn(1.f, g);
      if (r0 == 0 && ch == 0 && cv) reinterpret_cast<float*>(p.out + Lc.row_off())[c0 + c] = g;
    }
    uint32_t code[4];
#pragma unroll
    for (int b = 0; b < SPC; ++b) {
      float v[BLOCK];
      unsigned m = 0u;
#pragma unroll
      for (int e = 0; e < BLOCK; ++e) {
        v[e] = (float)tile[(ch * 32 + b * BLOCK + e) * 128 + c];
        m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
      }
      float mul = 0.f;
      bool zero;
      const uint8_t s = block_scale<BLOCK>(m, u, mul, zero);
      const int ks = ch * SPC + b;
      sfs[(ks >> 2) * 512 + (c & 31) * 16 + (c >> 5) * 4 + (ks & 3)] = s;
#pragma unroll
      for (int q = 0; q < BLOCK / 8; ++q) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __fmul_rn(v[q * 8 + e], mul);
        code[b * (BLOCK / 8) + q] = zero ? 0u : e2m1x8(w);
      }
    }
    *reinterpret_cast<uint4*>(p.out + tc * 8192 + ch * 2048 + c * 16) =
        make_uint4(code[0], code[1], code[2], code[3]);
  }
  __syncthreads();
  if (t < 32 * Lc.atoms())
    reinterpret_cast<uint4*>(p.out + Lc.scale_off() + tc * 512 * Lc.atoms())[t] =
        reinterpret_cast<const uint4*>(sfs)[t];
}

// ---------------------------------------------------------------------------
// Reading back: y[r][c] = code * block scale (* row scale), one CTA per tile.
// ---------------------------------------------------------------------------
// Eight codes to floats: code c is the fp16 value whose bits are the sign and
// c's three low bits moved to exponent and mantissa, times 2^14.
__device__ __forceinline__ void decode8(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = (w >> (4 * i)) & 15u;
    const float m = __half2float(__ushort_as_half((unsigned short)((c & 7u) << 9))) * 16384.f;
    v[i] = (c & 8u) ? -m : m;
  }
}

template <typename T, int BLOCK>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* packed, long long rows, long long cols, T* y,
                                                         int vec) {
  const Fp4Layout L(rows, cols, BLOCK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t ti = blockIdx.x;
  const int ty = blockIdx.x / (int)L.kt, tx = blockIdx.x - ty * (int)L.kt;
  const uint8_t* sf = packed + L.scale_off() + ti * 512 * L.atoms();
  for (int it = 0; it < 8; ++it) {
    const int item = it * 8 + warp, ch = item & 3, grp = item >> 2;
    const int rin = 8 * grp + (lane >> 2);
    const long long row = (long long)ty * 128 + rin;
    const long long k = (long long)tx * 128 + ch * 32 + (lane & 3) * 8;
    if (row >= rows || k >= cols) continue;
    const uint32_t w =
        *reinterpret_cast<const uint32_t*>(packed + ti * 8192 + ch * 2048 + rin * 16 + (lane & 3) * 4);
    const int ks = ch * (32 / BLOCK) + (BLOCK == 16 ? (lane & 3) >> 1 : 0);
    const uint8_t sb = sf[(ks >> 2) * 512 + (rin & 31) * 16 + (rin >> 5) * 4 + (ks & 3)];
    const float s = BLOCK == 16 ? e4m3_to_f(sb) : e8m0_to_f(sb);
    const float g = BLOCK == 16 ? reinterpret_cast<const float*>(packed + L.row_off())[row] : 1.f;
    float v[8];
    decode8(w, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = __fmul_rn(v[e], s);
      if (BLOCK == 16) v[e] = __fmul_rn(v[e], g);
    }
    T* out = y + row * cols + k;
    if (vec && k + 8 <= cols) {
      if (sizeof(T) == 2) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          o[i] = *reinterpret_cast<uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < cols) out[e] = (T)v[e];
    }
  }
}

template <typename T, int BLOCK>
cudaError_t launch_rows(const Fp4QuantArgs& a, cudaStream_t s) {
  const Fp4Layout L(a.rows, a.cols, BLOCK);
  const int threads = (int)std::min<long long>(512, std::max<long long>(128, L.kt * 4 * 32));
  quantize_rows_kernel<T, BLOCK><<<(unsigned)(L.rt * 16), threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int BLOCK>
cudaError_t launch_tiles(const Fp4QuantArgs& a, cudaStream_t s) {
  const Fp4Layout Lr(a.rows, a.cols, BLOCK), Lc(a.cols, a.rows, BLOCK);
  const unsigned grid = (unsigned)(Lr.kt * Lr.rt);
  cudaError_t e = cudaSuccess;
  if (BLOCK == 16) {
    unsigned* cm = reinterpret_cast<unsigned*>(a.out + Lc.max_off());
    unsigned* rm = a.out_rows ? reinterpret_cast<unsigned*>(a.out_rows + Lr.max_off()) : nullptr;
    e = cudaMemsetAsync(cm, 0, (size_t)Lc.rt * 512, s);
    if (e == cudaSuccess && rm) e = cudaMemsetAsync(rm, 0, (size_t)Lr.rt * 512, s);
    if (e != cudaSuccess) return e;
    absmax_kernel<T><<<grid, 256, 0, s>>>(a, cm, rm);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const size_t smem = 128 * 128 * sizeof(T);
  if (a.out_rows) {
    e = cudaFuncSetAttribute(quantize_tile_kernel<T, BLOCK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem);
    if (e != cudaSuccess) return e;
    quantize_tile_kernel<T, BLOCK, true><<<grid, 256, smem, s>>>(a);
  } else {
    e = cudaFuncSetAttribute(quantize_tile_kernel<T, BLOCK, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem);
    if (e != cudaSuccess) return e;
    quantize_tile_kernel<T, BLOCK, false><<<grid, 256, smem, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fp4

size_t fp4_packed_bytes(long long rows, long long cols, int block) { return Fp4Layout(rows, cols, block).bytes(); }

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, bool bf16, int block, bool rows_only, cudaStream_t s,
                                const char** kernel_name) {
  using namespace fp4;
  if (rows_only) {
    *kernel_name = "fp4_quantize_rows";
    if (bf16) return block == 16 ? launch_rows<__nv_bfloat16, 16>(a, s) : launch_rows<__nv_bfloat16, 32>(a, s);
    return block == 16 ? launch_rows<float, 16>(a, s) : launch_rows<float, 32>(a, s);
  }
  *kernel_name = a.out_rows ? (block == 16 ? "fp4_absmax+fp4_quantize_both" : "fp4_quantize_both")
                            : (block == 16 ? "fp4_absmax+fp4_quantize_columns" : "fp4_quantize_columns");
  if (bf16) return block == 16 ? launch_tiles<__nv_bfloat16, 16>(a, s) : launch_tiles<__nv_bfloat16, 32>(a, s);
  return block == 16 ? launch_tiles<float, 16>(a, s) : launch_tiles<float, 32>(a, s);
}

cudaError_t launch_fp4_dequantize(const void* packed, long long rows, long long cols, int block, void* y, bool bf16,
                                  cudaStream_t s, const char** kernel_name) {
  using namespace fp4;
  *kernel_name = "fp4_dequantize";
  const Fp4Layout L(rows, cols, block);
  const unsigned grid = (unsigned)(L.kt * L.rt);
  const uint8_t* in = static_cast<const uint8_t*>(packed);
  const int vec = (reinterpret_cast<uintptr_t>(y) % 16) == 0 && (cols * (bf16 ? 2 : 4)) % 16 == 0;
  if (bf16) {
    auto* o = static_cast<__nv_bfloat16*>(y);
    if (block == 16) dequantize_kernel<__nv_bfloat16, 16><<<grid, 256, 0, s>>>(in, rows, cols, o, vec);
    else dequantize_kernel<__nv_bfloat16, 32><<<grid, 256, 0, s>>>(in, rows, cols, o, vec);
  } else {
    auto* o = static_cast<float*>(y);
    if (block == 16) dequantize_kernel<float, 16><<<grid, 256, 0, s>>>(in, rows, cols, o, vec);
    else dequantize_kernel<float, 32><<<grid, 256, 0, s>>>(in, rows, cols, o, vec);
  }
  return cudaGetLastError();
}

}  // namespace qmm
