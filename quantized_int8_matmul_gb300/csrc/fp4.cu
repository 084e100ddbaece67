// Quantisation of a float matrix to 4-bit floats (e2m1) with block scales,
// along its rows, its columns, or both; and reading back.
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
// Bound by HBM: 0.53 or 0.56 bytes an element and direction are written, and x is read
// once with block 32, both ways too. With block 16 a row or column has to be whole
// before its first code: rows are read once where a CTA holds them, in registers (up to
// four steps a warp of bf16, two of float32) or in shared memory, else twice; columns
// once for up to 1024 rows (a cluster holds them), else twice, for their maxima and for
// their codes; both ways twice at least. A second reading comes from L2 as far as x fits.
#include "chain.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"

#include <algorithm>
#include <cuda_fp8.h>
#include <mutex>

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
  const uint8_t b = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  zero = !(t > 0.f) || !(u > 0.f) || b == 0;
  mul = __fdiv_rn(u, zero ? 1.f : e4m3_to_f(b));
  return zero ? 0 : b;
}

// Larger of each of two non-negative bf16 (a NaN wins), in one instruction.
constexpr uint32_t kMag = 0x7fff7fffu;   // magnitudes of two bf16
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (a * m, b * m), each rounded once, in one instruction.
__device__ __forceinline__ void mul_pair(float& a, float& b, float m) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(m));
}
__device__ __forceinline__ void mul8(float (&v)[8], float m) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) mul_pair(v[e], v[e + 1], m);
}

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 r;
  // elements [k, k + 8) of a row of n (k a multiple of 8; past the end: 0)
  __device__ __forceinline__ void load(const __nv_bfloat16* row, long long k, long long n, bool vec) {
    if (vec && k + 8 <= n) {
      r = *reinterpret_cast<const uint4*>(row + k);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* s = reinterpret_cast<const uint16_t*>(row) + k + 2 * i;
        w[i] = (k + 2 * i < n ? (uint32_t)s[0] : 0u) | (k + 2 * i + 1 < n ? (uint32_t)s[1] << 16 : 0u);
      }
      r = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void floats(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // bits of the largest magnitude as a float (a NaN is above infinity)
  __device__ __forceinline__ unsigned max_bits() const { return bits(pair()); }
  // the larger magnitudes of the even and of the odd elements, two bf16
  __device__ __forceinline__ uint32_t pair() const {
    return max_pair(max_pair(r.x & kMag, r.y & kMag), max_pair(r.z & kMag, r.w & kMag));
  }
  static __device__ __forceinline__ unsigned bits(uint32_t p) { return max(p << 16, p & 0xffff0000u); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, long long k, long long n, bool vec) {
    if (vec && k + 8 <= n) {
      a = *reinterpret_cast<const float4*>(row + k);
      b = *(reinterpret_cast<const float4*>(row + k) + 1);
    } else {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = k + e < n ? row[k + e] : 0.f;
      a = make_float4(v[0], v[1], v[2], v[3]);
      b = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __device__ __forceinline__ void floats(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ unsigned max_bits() const {
    float v[8];
    floats(v);
    unsigned m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    return m;
  }
};

// Sixteen consecutive elements, a lane's share of a row: a block of 16, or half a
// block of 32 (the other half in the neighbouring lane).
template <typename T>
struct Raw16 {
  Raw8<T> lo, hi;
  __device__ __forceinline__ void load(const T* row, long long k, long long n, bool vec) {
    lo.load(row, k, n, vec);
    hi.load(row, k + 8, n, vec);
  }
  __device__ __forceinline__ void load_whole(const T* p) {
    *this = *reinterpret_cast<const Raw16<T>*>(p);
  }
  // The same of global memory, where 32-byte alignment allows a whole sector a load
  // (half of one a load costs twice the requests).
  __device__ __forceinline__ void load_whole(const T* p, bool wide) {
    if (!wide) return load_whole(p);
    uint32_t* w = reinterpret_cast<uint32_t*>(this);
    const uint32_t* g = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < 4 * (int)sizeof(T); i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(g + i));
  }
  __device__ __forceinline__ unsigned max_bits() const {
    if constexpr (sizeof(T) == 2) return Raw8<T>::bits(max_pair(lo.pair(), hi.pair()));
    else return max(lo.max_bits(), hi.max_bits());
  }
  // the block's scale, and the elements' codes, the first in the lowest bits; m: max_bits()
  template <int BLOCK>
  __device__ __forceinline__ uint2 codes(unsigned m, float u, uint8_t& scale) const {
    if (BLOCK == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float mul = 0.f, f[8];
    bool zero;
    scale = block_scale<BLOCK>(m, u, mul, zero);
    uint2 c;
    lo.floats(f);
    mul8(f, mul);
    c.x = e2m1x8(f);
    hi.floats(f);
    mul8(f, mul);
    c.y = e2m1x8(f);
    return zero ? make_uint2(0u, 0u) : c;
  }
};

// A warp step's elements in shared memory, filled by neighbouring lanes from
// neighbouring columns; 16 bytes a row more keep the rows off each other's banks.
template <typename T, int ROWS, int COLS>
struct RowStage {
  static constexpr int PITCH = COLS + 16 / (int)sizeof(T);
  static constexpr int BYTES = ROWS * PITCH * (int)sizeof(T);
};

template <int J>
struct ScaleWord;   // J scale words of four
template <>
struct ScaleWord<4> { using type = uint4; };
template <>
struct ScaleWord<2> { using type = uint2; };
template <>
struct ScaleWord<1> { using type = uint32_t; };

// ---------------------------------------------------------------------------
// Along the rows. A CTA takes the rows {2c, 2c + 1} + 32 j of a tile, all four j
// (J = 4: a warp step is 64 columns of eight rows, 16 columns a lane), two of them
// (J = 2: 128 columns of four rows) or, for matrices of up to 32 rows, one (J = 1:
// 256 columns of two rows). Rows chosen so make every 32-byte sector of codes (two
// neighbouring rows' 16 bytes) the work of one CTA, and of scales (two rows'
// 16-byte lines of an atom, whose 4-byte parts are rows 32 apart) of one or two.
// Block 32 takes a segment of the columns a CTA (blockIdx.y). 8192 x 4096 bf16: block
// 32 14.9 us (5.7 TB/s, 85 % of a copy's rate), block 16 20.0 (64 %: a row has to be
// whole before its first code, so its loads, maximum and codes do not overlap within
// a CTA; the registers that hold it limit an SM to 32 warps). A warp's steps of a
// batch (ITER) are loaded together; with block 16 a row whose steps are one batch
// stays in registers between its maximum and its codes, longer rows are read again.
// ---------------------------------------------------------------------------
template <typename T, int BLOCK, int J, int ITER, bool VEC>
__global__ void __launch_bounds__(VEC ? 1024 : 896) quantize_rows_kernel(const Fp4QuantArgs p, const int staged,
                                                                                const int whole, const int turns) {
  constexpr int WROWS = 2 * J, WCOLS = 512 / WROWS;   // a warp step
  constexpr int ATOMS = BLOCK == 16 ? 2 : 1;
  constexpr int SPC = 32 / BLOCK;          // scales per 32-column chunk
  constexpr int LANES = 32 / WROWS;        // lanes a row
  constexpr int UC = LANES / 2;            // chunks a warp step
  __shared__ unsigned rowmax[8];
  const int nw = blockDim.x >> 5;
  // rows that no vector load can take: all of the CTA's rows (whole > 0: elements
  // between them), or a buffer a warp; then the scales (staged), [atom][2 rows][J
  // rows 32 apart][4]
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sfs = smem + (VEC ? 0 : whole ? WROWS * whole * (int)sizeof(T) : nw * RowStage<T, WROWS, WCOLS>::BYTES);
  chain_wait();
  const Fp4Layout L(p.rows, p.cols, BLOCK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_tile = J == 1 && p.rows <= 32 ? 16 : 64 / J;
  const int tile = blockIdx.x / per_tile, in_tile = blockIdx.x - tile * per_tile;
  const int c2 = 2 * (in_tile & 15), j0 = J * (in_tile >> 4);
  const int ri = lane / LANES, ra = ri & 1, rj = ri >> 1;
  const int piece = lane & (LANES - 1), half = piece & 1;
  const int rin = c2 + ra + 32 * (j0 + rj);
  const long long row = (long long)tile * 128 + rin, row_first = (long long)tile * 128 + c2 + 32 * j0;
  if (row_first >= p.rows) return;
  const bool rv = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + (rv ? row : 0) * p.ld;
  const int n = rv ? (int)p.cols : 0;
  const bool wide = ((reinterpret_cast<uintptr_t>(p.x) | (size_t)p.ld * sizeof(T)) & 31) == 0;
  const int chunks = (int)L.kt * 4, units_all = (chunks + UC - 1) / UC;
  // this CTA's steps: all, or (block 32) as many as its warps take in `turns` batches
  const int u0 = BLOCK == 32 && gridDim.y > 1 ? blockIdx.y * (nw * ITER * turns) : 0;
  const int units = BLOCK == 32 && gridDim.y > 1 ? min(units_all, u0 + nw * ITER * turns) : units_all;
  const int batches = (units - u0 + nw * ITER - 1) / (nw * ITER);
  if (!VEC && whole) {
    T* all = reinterpret_cast<T*>(smem);
    constexpr int CB = 16 / WROWS;   // 16 loads in flight: all rows, CB columns apart
    const T* xr[WROWS];
    int m[WROWS];
#pragma unroll
    for (int r = 0; r < WROWS; ++r) {
      const long long rr = row_first + (r & 1) + 32 * (r >> 1);
      xr[r] = static_cast<const T*>(p.x) + (rr < p.rows ? rr : 0) * p.ld;
      m[r] = rr < p.rows ? (int)p.cols : 0;
    }
    for (int c = threadIdx.x; c < units * WCOLS; c += CB * blockDim.x) {
      T e[CB][WROWS];
#pragma unroll
      for (int k = 0; k < CB; ++k)
#pragma unroll
        for (int r = 0; r < WROWS; ++r) {
          const int i = c + k * blockDim.x;
          e[k][r] = xr[r][min(i, (int)p.cols - 1)];
          if (i >= m[r]) e[k][r] = (T)0.f;
        }
#pragma unroll
      for (int k = 0; k < CB; ++k)
#pragma unroll
        for (int r = 0; r < WROWS; ++r) {
          const int i = c + k * blockDim.x;
          if (i < units * WCOLS) all[r * whole + i] = e[k][r];
        }
    }
    __syncthreads();
  }
  Raw16<T> v[ITER];
  auto load = [&](int b) {
    if (!VEC && whole) {
      const T* all = reinterpret_cast<const T*>(smem) + ri * whole + piece * 16;
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int un = (b * ITER + i) * nw + warp;
        if (un < units) v[i].load_whole(all + un * WCOLS);
        else v[i] = Raw16<T>{};
      }
      return;
    }
    if (VEC && (long long)(u0 + (b + 1) * ITER * nw) * WCOLS <= p.cols) {   // the whole batch lies inside
#pragma unroll
      for (int i = 0; i < ITER; ++i) v[i].load_whole(x + (u0 + (b * ITER + i) * nw + warp) * WCOLS + piece * 16, wide);
      return;
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {   // past the end: columns past n, zeros
      const long long k0 = (long long)(u0 + (b * ITER + i) * nw + warp) * WCOLS;
      if (VEC) {
        v[i].load(x, k0 + piece * 16, n, true);
      } else {
        using S = RowStage<T, WROWS, WCOLS>;
        T* buf = reinterpret_cast<T*>(smem + warp * S::BYTES);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < WROWS; ++r) {
          const long long rr = row_first + (r & 1) + 32 * (r >> 1);
          const T* xr = static_cast<const T*>(p.x) + (rr < p.rows ? rr : 0) * p.ld;
#pragma unroll
          for (int c = lane; c < WCOLS; c += 32)
            buf[r * S::PITCH + c] = rr < p.rows && k0 + c < p.cols ? xr[k0 + c] : (T)0.f;
        }
        __syncwarp();
        v[i] = *reinterpret_cast<const Raw16<T>*>(buf + ri * S::PITCH + piece * 16);
      }
    }
  };
  float u = 1.f;
  unsigned vm[ITER];
  if (BLOCK == 16) {
    if (threadIdx.x < 8) rowmax[threadIdx.x] = 0u;
    __syncthreads();
    unsigned m = 0u;
    for (int b = 0; b < batches; ++b) {
      load(b);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        vm[i] = v[i].max_bits();
        m = max(m, vm[i]);
      }
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (piece == 0) atomicMax(&rowmax[ri], m);
    __syncthreads();
    const float g = row_scale(rowmax[ri]);
    u = __fdiv_rn(1.f, g);
    if (warp == 0 && piece == 0 && rv) reinterpret_cast<float*>(p.out + L.row_off())[row] = g;
  }
  uint8_t* codes = p.out + (size_t)tile * L.kt * 8192 + rin * 16 + half * 8;
  uint8_t* sf = p.out + L.scale_off() + (size_t)tile * L.kt * 512 * ATOMS + c2 * 16 + j0 * 4;
  const int atom0 = u0 * UC * SPC / 4;   // the segment's first atom
  for (int b = 0; b < batches; ++b) {
    if (BLOCK == 32 || batches > 1) {
      load(b);
#pragma unroll
      for (int i = 0; i < ITER; ++i) vm[i] = v[i].max_bits();
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      uint8_t s;
      const uint2 code = v[i].template codes<BLOCK>(vm[i], u, s);
      const int ch = (u0 + (b * ITER + i) * nw + warp) * UC + (piece >> 1);
      if (ch < chunks) {
        const int k = ch * SPC + (BLOCK == 16 ? half : 0);
        const bool mine = BLOCK == 16 || half == 0;
        if (rv) *reinterpret_cast<uint2*>(codes + (size_t)ch * 2048) = code;
        if (mine && staged) sfs[((k >> 2) - atom0) * (8 * J) + ra * 4 * J + rj * 4 + (k & 3)] = s;
        if (mine && !staged && rv) sf[(size_t)(k >> 2) * 512 + ra * 16 + rj * 4 + (k & 3)] = s;
      }
    }
  }
  chain_release();
  if (staged) {   // a row's J scale words of an atom at a time
    __syncthreads();
    using Word = typename ScaleWord<J>::type;
    const int atoms = (min(chunks, units * UC) * SPC + 3) / 4 - atom0;
    for (int i = threadIdx.x; i < atoms * 2; i += blockDim.x)
      *reinterpret_cast<Word*>(sf + (size_t)(atom0 + (i >> 1)) * 512 + (i & 1) * 16) =
          reinterpret_cast<const Word*>(sfs)[i];
  }
}

// The same for block 16 and many long rows: a ring of groups of rows (J = 1: two
// rows each) filled by bulk copies, so that the next groups are on their way while
// one waits for its rows' maxima and is turned into codes. A group is read from
// shared memory twice, its blocks' maxima stay in registers. 4096 x 11008 bf16:
// 26.8 us (4.3 TB/s, 64 % of a copy's rate).
// Waits are bounded (common.cuh).
constexpr int RING_THREADS = 512, RING_STEPS = 4, RING_MAX = 8;
constexpr unsigned SITE_ROWS = 0x530;
__global__ void __launch_bounds__(RING_THREADS, 2) quantize_rows_ring_kernel(const Fp4QuantArgs p, const int groups,
                                                                            const int slots, const uint32_t pitch) {
  using T = __nv_bfloat16;
  constexpr int J = 1, WROWS = 2 * J, WCOLS = 512 / WROWS, LANES = 32 / WROWS, UC = LANES / 2, NW = RING_THREADS / 32;
  constexpr int PER_TILE = 64 / J;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned rowmax[2][8];
  __shared__ uint64_t full[RING_MAX];
  chain_wait();
  const Fp4Layout L(p.rows, p.cols, 16);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int ri = lane / LANES, ra = ri & 1, rj = ri >> 1, piece = lane & (LANES - 1), half = piece & 1;
  const int chunks = (int)L.kt * 4, units = (chunks + UC - 1) / UC, atoms = (int)L.kt * 2;
  const uint32_t line = (uint32_t)p.cols * (uint32_t)sizeof(T);   // a row's bytes
  uint8_t* sfs = smem + (size_t)slots * WROWS * pitch;   // two groups' scales
  auto first_row = [&](int g) {
    const int tile = g / PER_TILE, in = g - tile * PER_TILE;
    return (long long)tile * 128 + 2 * (in & 15) + 32 * J * (in >> 4);
  };
  auto fill = [&](int k) {   // one thread: the CTA's k-th group
    const long long r0 = first_row(blockIdx.x + k * gridDim.x);
    uint64_t* bar = &full[k % slots];
    uint32_t bytes = 0u;
#pragma unroll
    for (int r = 0; r < WROWS; ++r)
      if (r0 + (r & 1) + 32 * (r >> 1) < p.rows) bytes += line;
    mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int r = 0; r < WROWS; ++r) {
      const long long row = r0 + (r & 1) + 32 * (r >> 1);
      if (row < p.rows)
        bulk_load(smem_u32(smem) + (uint32_t)((k % slots) * WROWS + r) * pitch, static_cast<const T*>(p.x) + row * p.ld,
                  line, bar);
    }
  };
  const int mine = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  if (t < 8) rowmax[0][t] = 0u;
  if (t == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
    for (int k = 0; k < slots && k < mine; ++k) fill(k);
  }
  __syncthreads();
  for (int k = 0; k < mine; ++k) {
    const int slot = k % slots;
    if (!mbar_wait(&full[slot], (uint32_t)((k / slots) & 1), nullptr, p.err, SITE_ROWS)) {
      // (the copies of the later slots are waited for, with the same limit, before the CTA ends)
      for (int i = 1; i < slots && k + i < mine; ++i)
        mbar_wait(&full[(k + i) % slots], (uint32_t)(((k + i) / slots) & 1), nullptr, p.err, SITE_ROWS);
      break;
    }
    const int g = blockIdx.x + k * gridDim.x, tile = g / PER_TILE, in = g - tile * PER_TILE;
    const int c2 = 2 * (in & 15), j0 = J * (in >> 4), rin = c2 + ra + 32 * (j0 + rj);
    const long long row = (long long)tile * 128 + rin;
    const bool rv = row < p.rows;
    const T* x = reinterpret_cast<const T*>(smem + (size_t)(slot * WROWS + ri) * pitch);
    const int n = rv ? (int)p.cols : 0;
    auto get = [&](int un) {   // zeros past the end
      const int c = un * WCOLS + piece * 16;
      Raw16<T> v;
      if (c + 16 <= n) v.load_whole(x + c);
      else v.load(x, c, n, true);
      return v;
    };
    unsigned m = 0u, vm[RING_STEPS];
#pragma unroll
    for (int i = 0; i < RING_STEPS; ++i) {
      vm[i] = 0u;
      if (warp + i * NW < units) vm[i] = get(warp + i * NW).max_bits();
      m = max(m, vm[i]);
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (piece == 0) atomicMax(&rowmax[k & 1][ri], m);
    __syncthreads();
    const float gs = row_scale(rowmax[k & 1][ri]), u = __fdiv_rn(1.f, gs);
    if (warp == 0 && piece == 0 && rv) reinterpret_cast<float*>(p.out + L.row_off())[row] = gs;
    if (t < 8) rowmax[(k + 1) & 1][t] = 0u;
    uint8_t* codes = p.out + (size_t)tile * L.kt * 8192 + rin * 16 + half * 8;
    uint8_t* ss = sfs + (size_t)(k & 1) * atoms * 8 * J + ra * 4 * J + rj * 4;
#pragma unroll
    for (int i = 0; i < RING_STEPS; ++i) {
      const int un = warp + i * NW, ch = un * UC + (piece >> 1);
      if (un < units) {
        uint8_t sc;
        const uint2 code = get(un).template codes<16>(vm[i], u, sc);
        if (ch < chunks) {
          const int ks = ch * 2 + half;
          if (rv) *reinterpret_cast<uint2*>(codes + (size_t)ch * 2048) = code;
          ss[(ks >> 2) * (8 * J) + (ks & 3)] = sc;
        }
      }
    }
    __syncthreads();
    if (t == 0 && k + slots < mine) {
      fence_proxy_async_smem();   // the slot was read through the generic proxy
      fill(k + slots);
    }
    using Word = typename ScaleWord<J>::type;   // a row's J scale words of an atom at a time
    uint8_t* sf = p.out + L.scale_off() + (size_t)tile * L.kt * 1024 + c2 * 16 + j0 * 4;
    const Word* from = reinterpret_cast<const Word*>(sfs + (size_t)(k & 1) * atoms * 8 * J);
    for (int i = t; i < atoms * 2; i += RING_THREADS)
      *reinterpret_cast<Word*>(sf + (size_t)(i >> 1) * 512 + (i & 1) * 16) = from[i];
  }
}

// a[0 .. na) and b[0 .. n - na) to zero, before the maxima: two fills of the
// library's took 2 us longer, as they do not start on the heels of what precedes them.
__global__ void __launch_bounds__(256) zero_kernel(unsigned* a, long long na, unsigned* b, long long n) {
  chain_wait();
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  if (i < na) a[i] = 0u;
  else if (i < n) b[i - na] = 0u;
  chain_release();
}


// ---------------------------------------------------------------------------
// Along the columns, or both ways: x is [rows][cols] in memory; the packed
// matrix along the columns is its transpose [cols][rows].
// ---------------------------------------------------------------------------
// Largest magnitudes of the columns (and the rows) into the packed buffers' max
// words: 64 rows x 256 columns a CTA, eight columns a lane. 8192 x 4096 bf16: 11 of
// the 26.7 us that block 16 takes along the columns (the second reading of x is
// largely from L2).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 4 : 2) absmax_kernel(const Fp4QuantArgs p, unsigned* colmax,
                                                                  unsigned* rowmax) {
  __shared__ unsigned cm[256];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ct = (int)((p.cols + 255) / 256), ty = blockIdx.x / ct, tx = blockIdx.x - ty * ct;
  const long long c = (long long)tx * 256, r0 = (long long)ty * 64 + warp;
  cm[threadIdx.x] = 0u;
  __syncthreads();
  // rows past the end read the last one again: no maximum changes
  const T* x = static_cast<const T*>(p.x);
  if (VEC && c + 256 <= p.cols) {
    constexpr int CW = 4 / sizeof(T), NWORD = 8 / CW;   // 32-bit words of a lane's eight columns
    constexpr int NB = 16 / (int)sizeof(T);               // rows in flight
    uint32_t m[NWORD] = {};
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += NB) {
      Raw8<T> v[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i)
        v[i] = *reinterpret_cast<const Raw8<T>*>(x + min(r0 + 8 * (i0 + i), p.rows - 1) * p.ld + c + lane * 8);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[i]);
#pragma unroll
        for (int e = 0; e < NWORD; ++e) m[e] = CW == 2 ? max_pair(m[e], w[e] & kMag) : max(m[e], w[e] & 0x7fffffffu);
        if (rowmax) {
          const unsigned rm = __reduce_max_sync(0xffffffffu, v[i].max_bits());
          if (lane == 0 && r0 + 8 * (i0 + i) < p.rows) atomicMax(rowmax + r0 + 8 * (i0 + i), rm);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = m[e / CW];
      atomicMax(&cm[lane * 8 + e], CW == 1 ? w : (e & 1) ? w & 0xffff0000u : w << 16);
    }
  } else {   // neighbouring lanes, neighbouring columns (past the end the last one again)
    unsigned m[8] = {};
    constexpr int NB = VEC ? 2 : 8;   // (VEC: the last columns alone)
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += NB) {
      T v[NB][8];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const T* row = x + min(r0 + 8 * (i0 + i), p.rows - 1) * p.ld;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = row[min(c + e * 32 + lane, p.cols - 1)];
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        unsigned rm = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const unsigned b = __float_as_uint((float)v[i][e]) & 0x7fffffffu;
          m[e] = max(m[e], b);
          rm = max(rm, b);
        }
        if (rowmax) {
          rm = __reduce_max_sync(0xffffffffu, rm);
          if (lane == 0 && r0 + 8 * (i0 + i) < p.rows) atomicMax(rowmax + r0 + 8 * (i0 + i), rm);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) atomicMax(&cm[e * 32 + lane], m[e]);
  }
  chain_release();
  __syncthreads();
  if (c + threadIdx.x < p.cols) atomicMax(colmax + c + threadIdx.x, cm[threadIdx.x]);
}

// One tile of 128 x 128 of x a CTA: its rows are quantised as they are loaded
// (ROWS), all of it goes to shared memory, and its columns are quantised from
// there. The scales leave as whole tiles by bulk copies. CLUSTER (block 16,
// x of up to 8 tiles down): the tiles above each other are one cluster, and the
// columns' maxima are taken over it -- one launch in place of a fill, a pass for
// the maxima and this. 8192 x 4096 bf16: block 32 both ways 19.6 us (5.3 TB/s, 79 %
// of a copy's rate; issue slots 56 % busy), columns alone 15.1; block 16 with its
// maxima 36.2 and 26.7. 4099 x 1021 float32, block 16, columns: 8.4 us.
template <typename T>
struct TileSmem {
  static constexpr int PITCH = 128 * (int)sizeof(T) + 16;   // bytes; 16 more keep row accesses off each other's banks
  static constexpr int SCALES = 128 * PITCH;                // two tiles of scales
  static constexpr int BYTES = SCALES + 2 * 1024;
};

template <typename T, int BLOCK, bool ROWS, bool CLUSTER>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 5 : 3) quantize_tile_kernel(const Fp4QuantArgs p) {
  chain_wait();
  using S = TileSmem<T>;
  constexpr int ATOMS = BLOCK == 16 ? 2 : 1;
  constexpr int SPC = 32 / BLOCK;
  constexpr int CW = 4 / sizeof(T);   // columns in a 32-bit word
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sf_c = smem + S::SCALES;
  uint8_t* sf_r = sf_c + 1024;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const Fp4Layout Lr(p.rows, p.cols, BLOCK), Lc(p.cols, p.rows, BLOCK);
  const int across = CLUSTER ? (int)Lr.rt : (int)Lr.kt;
  const int b1 = blockIdx.x / across, b0 = blockIdx.x - b1 * across;
  const int ty = CLUSTER ? b0 : b1, tx = CLUSTER ? b1 : b0;
  const long long c0 = (long long)tx * 128, r0 = (long long)ty * 128;
  const size_t ti = (size_t)ty * Lr.kt + tx;          // this tile in the packed rows
  const size_t tc = (size_t)tx * Lc.kt + ty;          // and in the packed columns
  // a warp step: 8 rows x 64 columns; warp w takes rows 8w .. 8w + 7 of each 64
  Raw16<T> v[4];
  const int half = lane & 1;
  if (!p.vec) {   // neighbouring lanes, neighbouring columns, into shared memory first
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const long long r = r0 + i * 8 + warp;
      const T* x = static_cast<const T*>(p.x) + (r < p.rows ? r : 0) * p.ld;
      T* d = reinterpret_cast<T*>(smem + (i * 8 + warp) * S::PITCH);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long c = c0 + j * 32 + lane;
        d[j * 32 + lane] = r < p.rows && c < p.cols ? x[c] : (T)0.f;
      }
    }
    __syncthreads();
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(p.x) | (size_t)p.ld * sizeof(T)) & 31) == 0;
  const bool inside = p.vec && r0 + 128 <= p.rows && c0 + 128 <= p.cols;
  if (inside) {
    const T* x = static_cast<const T*>(p.x) + (r0 + warp * 8 + (lane >> 2)) * p.ld + c0 + (lane & 3) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].load_whole(x + (i >> 1) * 64 * p.ld + (i & 1) * 64, wide);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (inside) break;
    const int rin = (i >> 1) * 64 + warp * 8 + (lane >> 2), k = (i & 1) * 64 + (lane & 3) * 16;
    const bool rv = r0 + rin < p.rows;
    if (p.vec)
      v[i].load(static_cast<const T*>(p.x) + (rv ? r0 + rin : 0) * p.ld, c0 + k, rv ? p.cols : 0, true);
    else if (ROWS)
      v[i] = *reinterpret_cast<const Raw16<T>*>(smem + rin * S::PITCH + k * sizeof(T));
  }
  float u = 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rin = (i >> 1) * 64 + warp * 8 + (lane >> 2), k = (i & 1) * 64 + (lane & 3) * 16;
    if (p.vec) *reinterpret_cast<Raw16<T>*>(smem + rin * S::PITCH + k * sizeof(T)) = v[i];
    if (ROWS) {
      if (BLOCK == 16 && (i & 1) == 0) {
        const bool rv = r0 + rin < p.rows;
        const float g = row_scale(rv ? reinterpret_cast<const unsigned*>(p.out_rows + Lr.max_off())[r0 + rin] : 0u);
        u = __fdiv_rn(1.f, g);
        if (c0 == 0 && (lane & 3) == 0 && rv) reinterpret_cast<float*>(p.out_rows + Lr.row_off())[r0 + rin] = g;
      }
      uint8_t s;
      const uint2 code = v[i].template codes<BLOCK>(v[i].max_bits(), u, s);
      const int ch = k >> 5, ks = ch * SPC + (BLOCK == 16 ? half : 0);
      // (8 rows of a chunk: 128 bytes of the packed tile)
      *reinterpret_cast<uint2*>(p.out_rows + ti * 8192 + ch * 2048 + rin * 16 + half * 8) = code;
      if (BLOCK == 16 || half == 0) sf_r[(ks >> 2) * 512 + (rin & 31) * 16 + (rin >> 5) * 4 + (ks & 3)] = s;
    }
  }
  __syncthreads();
  __shared__ unsigned cmax[CLUSTER ? 128 : 1];   // this tile's, then read by the cluster
  unsigned* call = reinterpret_cast<unsigned*>(sf_r);   // the whole columns'
  if (CLUSTER) {
    if (t < 128) cmax[t] = 0u;
    __syncthreads();
    for (int item = t; item < 4 * 128 / CW; item += 256) {
      const int cw = item % (128 / CW), ch = item / (128 / CW);
      uint32_t m = 0u;
#pragma unroll 8
      for (int e = 0; e < 32; ++e) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(smem + (ch * 32 + e) * S::PITCH + cw * 4);
        m = CW == 2 ? max_pair(m, x & kMag) : max(m, x & 0x7fffffffu);
      }
      if (CW == 2) {
        atomicMax(&cmax[2 * cw], m << 16);
        atomicMax(&cmax[2 * cw + 1], m & 0xffff0000u);
      } else {
        atomicMax(&cmax[cw], m);
      }
    }
    cluster_sync_all();
    if (t < 128) {
      unsigned m = 0u;
      for (int r = 0; r < (int)Lr.rt; ++r) {
        uint32_t x;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(mapa_shared(smem_u32(&cmax[t]), (uint32_t)r)));
        m = max(m, x);
      }
      call[t] = m;
    }
    cluster_sync_all();   // (the others have read cmax)
  }
  const bool wide_out = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;   // (16-byte alignment is all that is asked)
  // a work item: 32 rows of the column(s) in one 32-bit word
#pragma unroll 1
  for (int item = t; item < 4 * 128 / CW; item += 256) {
    const int cw = item % (128 / CW), ch = item / (128 / CW);
    float uc[CW];
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      uc[w] = 1.f;
      if (BLOCK == 16) {
        const long long c = c0 + cw * CW + w;
        const float g = row_scale(CLUSTER ? call[cw * CW + w]
                                  : c < p.cols ? reinterpret_cast<const unsigned*>(p.out + Lc.max_off())[c] : 0u);
        uc[w] = __fdiv_rn(1.f, g);
        if (r0 == 0 && ch == 0 && c < p.cols) reinterpret_cast<float*>(p.out + Lc.row_off())[c] = g;
      }
    }
    uint32_t code[CW][4];
#pragma unroll
    for (int b = 0; b < SPC; ++b) {
      uint32_t x[BLOCK], m = 0u;
#pragma unroll
      for (int e = 0; e < BLOCK; ++e) {
        x[e] = *reinterpret_cast<const uint32_t*>(smem + (ch * 32 + b * BLOCK + e) * S::PITCH + cw * 4);
        m = CW == 2 ? max_pair(m, x[e] & kMag) : max(m, x[e] & 0x7fffffffu);
      }
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const unsigned mb = CW == 1 ? m : w == 0 ? m << 16 : m & 0xffff0000u;
        float mul = 0.f;
        bool zero;
        const uint8_t s = block_scale<BLOCK>(mb, uc[w], mul, zero);
        const int ks = ch * SPC + b, c = cw * CW + w;
        sf_c[(ks >> 2) * 512 + (c & 31) * 16 + (c >> 5) * 4 + (ks & 3)] = s;
#pragma unroll
        for (int q = 0; q < BLOCK / 8; ++q) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t xe = x[q * 8 + e];
            f[e] = __uint_as_float(CW == 1 ? xe : w == 0 ? xe << 16 : xe & 0xffff0000u);
          }
          mul8(f, mul);
          code[w][b * (BLOCK / 8) + q] = zero ? 0u : e2m1x8(f);
        }
      }
    }
    uint8_t* d = p.out + tc * 8192 + ch * 2048 + cw * CW * 16;
    if (CW == 2 && wide_out) {   // two columns' codes as one store
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "r"(code[0][0]),
                   "r"(code[0][1]), "r"(code[0][2]), "r"(code[0][3]), "r"(code[CW - 1][0]), "r"(code[CW - 1][1]),
                   "r"(code[CW - 1][2]), "r"(code[CW - 1][3])
                   : "memory");
    } else {
#pragma unroll
      for (int w = 0; w < CW; ++w)
        reinterpret_cast<uint4*>(d)[w] = make_uint4(code[w][0], code[w][1], code[w][2], code[w][3]);
    }
  }
  chain_release();
  fence_proxy_async_smem();   // this thread's writes, visible to the copy engine
  __syncthreads();
  if (t == 0) {
    bulk_store(p.out + Lc.scale_off() + tc * (512 * ATOMS), smem_u32(sf_c), 512 * ATOMS);
    if (ROWS) {
      bulk_store(p.out_rows + Lr.scale_off() + ti * (512 * ATOMS), smem_u32(sf_r), 512 * ATOMS);
    }
    bulk_commit();
    bulk_wait_all();
  }
}

// ---------------------------------------------------------------------------
// Reading back: y[r][c] = code * block scale (* row scale), one CTA per tile.
// 8192 x 4096 to bf16 14.2 us (6.0 TB/s, 90 % of a copy's rate); 4099 x 1021 to
// float32, whose rows start off 16 bytes, 5.2 us (3.7 TB/s).
// ---------------------------------------------------------------------------
// Eight codes, the first in the lowest bits, by the conversion to fp16 pairs.
__device__ __forceinline__ void decode8(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\tcvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}

template <typename T, int BLOCK, bool VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* packed, long long rows, long long cols, T* y) {
  chain_wait();
  constexpr int ATOMS = BLOCK == 16 ? 2 : 1;
  const Fp4Layout L(rows, cols, BLOCK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t ti = blockIdx.x;
  const int ty = blockIdx.x / (int)L.kt, tx = blockIdx.x - ty * (int)L.kt;
  const uint8_t* codes = packed + ti * 8192;
  const uint8_t* sf = packed + L.scale_off() + ti * (512 * ATOMS);
  const float* gs = reinterpret_cast<const float*>(packed + L.row_off()) + (long long)ty * 128;
  const long long r0 = (long long)ty * 128, c0 = (long long)tx * 128;
  // 8 rows x 32 columns a warp step, eight columns a lane
  const bool wide = ((reinterpret_cast<uintptr_t>(y) | (size_t)cols * sizeof(T)) & 31) == 0;
  uint32_t w[8];
  uint8_t sb[8];
  float g[2] = {1.f, 1.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = i & 3, rin = (i >> 2) * 64 + warp * 8 + (lane >> 2);
    const int ks = ch * (32 / BLOCK) + (BLOCK == 16 ? (lane & 3) >> 1 : 0);
    w[i] = *reinterpret_cast<const uint32_t*>(codes + ch * 2048 + rin * 16 + (lane & 3) * 4);
    sb[i] = sf[(ks >> 2) * 512 + (rin & 31) * 16 + (rin >> 5) * 4 + (ks & 3)];
    if (BLOCK == 16 && ch == 0 && r0 + rin < rows) g[i >> 2] = gs[rin];
  }
  chain_release();
  // rows that start off 16 bytes: a warp's eight rows through shared memory, then a
  // row at a time, neighbouring lanes neighbouring elements
  constexpr int PITCH = 128 + 16 / (int)sizeof(T);
  __shared__ __align__(16) T rows_s[VEC ? 1 : 8 * 8 * PITCH];
  T* buf = rows_s + (VEC ? 0 : warp * 8 * PITCH);
  const int n = (int)min(128ll, cols - c0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = i & 3, rin = (i >> 2) * 64 + warp * 8 + (lane >> 2);
    const long long row = r0 + rin, k = c0 + ch * 32 + (lane & 3) * 8;
    const float s = BLOCK == 16 ? e4m3_to_f(sb[i]) : e8m0_to_f(sb[i]);
    float v[8];
    decode8(w[i], v);
    mul8(v, s);
    if (BLOCK == 16) mul8(v, g[i >> 2]);
    // cols is a multiple of 16 bytes (VEC): 8 columns lie inside, or 4 of float32
    T* out = VEC ? y + row * cols + k : buf + (lane >> 2) * PITCH + ch * 32 + (lane & 3) * 8;
    if (!VEC || (row < rows && k < cols)) {
      if (sizeof(T) == 2) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          o[e] = *reinterpret_cast<uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
      } else if (VEC && wide && k + 4 < cols) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(v[0]), "f"(v[1]),
                     "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
      } else {
        reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
        if (!VEC || k + 4 < cols) reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    if (VEC || ch < 3) continue;
    __syncwarp();
    const long long first = r0 + (i >> 2) * 64 + warp * 8;
    const int some = (int)max(0ll, min(8ll, rows - first));
#pragma unroll 4
    for (int r = 0; r < some; ++r) {
      T* d = y + (first + r) * cols + c0;
      const T* from = buf + r * PITCH;
      if (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j * 32 + lane < n) d[j * 32 + lane] = from[j * 32 + lane];
      } else {   // pairs of bf16 from the first 4-byte boundary on
        const int odd = (int)(reinterpret_cast<uintptr_t>(d) >> 1) & 1;
        if (odd && lane == 0) d[0] = from[0];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = odd + j * 64 + 2 * lane;
          if (e + 1 < n) {
            const uint32_t lo = reinterpret_cast<const uint16_t*>(from)[e];
            const uint32_t hi = reinterpret_cast<const uint16_t*>(from)[e + 1];
            *reinterpret_cast<uint32_t*>(d + e) = lo | hi << 16;
          } else if (e < n) {
            d[e] = from[e];
          }
        }
      }
    }
    __syncwarp();
  }
}

// Steps a warp loads together and warps a CTA. Block 16: as few CTAs' rows as fill
// the registers of one batch, four steps of bf16 or two of float32 (64 registers a
// thread); block 32: four warps of them, the columns over as many CTAs as it takes.
template <typename T, int BLOCK, int J>
cudaError_t launch_rows_j(const Fp4QuantArgs& a, cudaStream_t s) {
  constexpr int WROWS = 2 * J, WCOLS = 512 / WROWS, MOST = sizeof(T) == 2 ? 4 : 2;
  const Fp4Layout L(a.rows, a.cols, BLOCK);
  const long long units = (L.kt * 128 + WCOLS - 1) / WCOLS;
  const unsigned grid = (unsigned)(J == 1 && a.rows <= 32 ? 16 : L.rt * (64 / J));
  size_t smem = (size_t)L.kt * L.atoms() * 8 * J;
  int staged = smem <= (a.vec ? 40 : 16) * 1024;
  if (!staged) smem = 0;
  if (!a.vec) {
    auto kern = quantize_rows_kernel<T, BLOCK, J, 2, false>;
    static std::once_flag once[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev],
                   [&] { e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024); });
    if (e != cudaSuccess) return e;
    // all rows in shared memory (16 bytes a row more keep them off each other's
    // banks), or, where they are too long, the warps' buffers
    const long long whole = units * WCOLS + 16 / (long long)sizeof(T);
    if (whole * WROWS * (long long)sizeof(T) + (long long)smem <= 200 * 1024) {
      const int nw = (int)std::min<long long>(16, std::max<long long>(8, (units + 1) / 2));
      return launch_chained(kern, grid, nw * 32, smem + (size_t)whole * WROWS * sizeof(T), 1, s, a, staged, (int)whole,
                            1);
    }
    const int nw = 28;
    return launch_chained(kern, grid, nw * 32, smem + (size_t)nw * RowStage<T, WROWS, WCOLS>::BYTES, 1, s, a, staged, 0,
                          1);
  }
  int iter = 1;   // (a CTA alone on its SM takes more warps)
  while (iter < MOST && units > (BLOCK == 32 ? 4 : (int)grid < num_sms() ? 16 : 8) * iter) iter *= 2;
  int nw = (int)std::min<long long>(32, std::max<long long>(4, (units + iter - 1) / iter));
  // a segment is one batch, or as many as keep the segments on their grid axis (65,535:
  // above 33 million columns of float32 in more than 32 rows, 67 of bf16)
  constexpr long long AXIS = 65535;
  unsigned segments = 1;
  int turns = 1;
  if (BLOCK == 32 && units > 4 * iter) {
    nw = 4;
    turns = (int)((units + 4 * iter * AXIS - 1) / (4 * iter * AXIS));
    segments = (unsigned)((units + 4 * iter * turns - 1) / (4 * iter * turns));
    smem = (size_t)(4 * iter * turns * WCOLS / 128) * 8 * J;
    staged = 1;
  }
  auto kern = iter == 1   ? quantize_rows_kernel<T, BLOCK, J, 1, true>
              : iter == 2 ? quantize_rows_kernel<T, BLOCK, J, 2, true>
                          : quantize_rows_kernel<T, BLOCK, J, MOST, true>;
  return launch_chained(kern, dim3(grid, segments), nw * 32, smem, 1, s, a, staged, 0, turns);
}

// Long bf16 rows by the ring, where two groups of two rows leave room for a second
// CTA on the SM and there are groups for two rounds. 4096 x 11008: 35.0 us without,
// 26.9 with; 2000 x 12288 19.4 and 17.9. The two barriers a group cost shorter rows
// more than they gain (4096 x 8192: 22.9 and 22.5; 8192 x 4096: 20.0 and 21.8 at
// best), and float32 rows, half as many elements a slot (1531 x 6144: 14.7 and 16.6).
bool launch_rows_ring(const Fp4QuantArgs& a, cudaStream_t s, cudaError_t& e) {
  using T = __nv_bfloat16;
  const Fp4Layout L(a.rows, a.cols, 16);
  const long long row = a.cols * (long long)sizeof(T);
  if (!a.vec || row % 16 != 0 || row <= 16 * 1024 || a.rows < 8 * num_sms()) return false;
  const uint32_t pitch = (uint32_t)row + 16;   // (keeps the rows off each other's banks)
  const int slots = (int)std::min<long long>(RING_MAX, (106 * 1024 - L.kt * 32) / (2ll * pitch));
  if (slots < 2 || L.kt * 128 > RING_STEPS * (RING_THREADS / 32) * 256) return false;
  auto kern = quantize_rows_ring_kernel;
  static std::once_flag once[64];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return true;
  std::call_once(once[dev],
                 [&] { e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 * 1024); });
  if (e != cudaSuccess) return true;
  const int groups = (int)(L.rt * 64);
  e = launch_chained(kern, (unsigned)std::min(groups, 2 * num_sms()), RING_THREADS,
                     (size_t)slots * 2 * pitch + (size_t)L.kt * 32, 1, s, a, groups, slots, pitch);
  return true;
}

template <typename T, int BLOCK>
cudaError_t launch_rows(const Fp4QuantArgs& a, cudaStream_t s) {
  if (BLOCK == 16 && sizeof(T) == 2) {
    cudaError_t e = cudaSuccess;
    if (launch_rows_ring(a, s, e)) return e;
  }
  // Two rows a CTA where more would not give every SM one (137 x 4100 bf16, block 16:
  // 5.2 us with four, 3.8 with two; block 32 of aligned rows has its segments
  // instead), or where four would be too long for two CTAs' registers on an SM and the
  // ring does not apply (1000 x 11008 and the like; 4096 x 11008 38.8 and 35.4).
  const bool few = (a.rows + 127) / 128 * 32 < num_sms();
  if constexpr (BLOCK == 32) {
    if (a.rows <= 32 || (few && !a.vec)) return launch_rows_j<T, BLOCK, 1>(a, s);
    return launch_rows_j<T, BLOCK, 4>(a, s);
  } else {
    if (few || (a.vec && a.cols > 8192)) return launch_rows_j<T, BLOCK, 1>(a, s);
    return launch_rows_j<T, BLOCK, 2>(a, s);
  }
}

template <typename T, int BLOCK, bool ROWS, bool CLUSTER>
cudaError_t launch_tile(const Fp4QuantArgs& a, unsigned grid, unsigned cluster, cudaStream_t s) {
  static std::once_flag once[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kern = quantize_tile_kernel<T, BLOCK, ROWS, CLUSTER>;
  std::call_once(once[dev], [&] {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TileSmem<T>::BYTES);
  });
  if (e != cudaSuccess) return e;
  return launch_chained(kern, grid, 256, TileSmem<T>::BYTES, cluster, s, a);
}

// Block 16, x of up to 8 tiles down: the columns by clusters, the rows (both ways)
// by their own kernel.
inline bool by_clusters(const Fp4QuantArgs& a, int block) { return block == 16 && a.rows <= 8 * 128; }

template <typename T, int BLOCK>
cudaError_t launch_tiles(const Fp4QuantArgs& a, cudaStream_t s) {
  const Fp4Layout Lr(a.rows, a.cols, BLOCK), Lc(a.cols, a.rows, BLOCK);
  const unsigned grid = (unsigned)(Lr.kt * Lr.rt);
  if (BLOCK == 16 && by_clusters(a, BLOCK)) {
    if (a.out_rows) {
      Fp4QuantArgs r = a;
      r.out = a.out_rows;
      r.out_rows = nullptr;
      const cudaError_t e = launch_rows<T, BLOCK>(r, s);
      if (e != cudaSuccess) return e;
    }
    return launch_tile<T, BLOCK, false, BLOCK == 16>(a, grid, (unsigned)Lr.rt, s);
  }
  if (BLOCK == 16) {
    unsigned* cm = reinterpret_cast<unsigned*>(a.out + Lc.max_off());
    unsigned* rm = a.out_rows ? reinterpret_cast<unsigned*>(a.out_rows + Lr.max_off()) : nullptr;
    const long long cols = Lc.rt * 128, words = cols + (rm ? Lr.rt * 128 : 0);   // (together past 2^31)
    cudaError_t e = launch_chained(zero_kernel, (unsigned)((words + 255) / 256), 256, 0, 1, s, cm, cols, rm, words);
    if (e != cudaSuccess) return e;
    const long long ctas = ((a.cols + 255) / 256) * ((a.rows + 63) / 64);
    e = launch_chained(a.vec ? absmax_kernel<T, true> : absmax_kernel<T, false>, (unsigned)ctas, 256, 0, 1, s, a, cm,
                       rm);
    if (e != cudaSuccess) return e;
  }
  return a.out_rows ? launch_tile<T, BLOCK, true, false>(a, grid, 1, s)
                    : launch_tile<T, BLOCK, false, false>(a, grid, 1, s);
}

template <typename T, int BLOCK>
cudaError_t launch_dequantize(const uint8_t* in, long long rows, long long cols, void* y, cudaStream_t s) {
  const Fp4Layout L(rows, cols, BLOCK);
  const unsigned grid = (unsigned)(L.kt * L.rt);
  const bool vec = (reinterpret_cast<uintptr_t>(y) % 16) == 0 && (cols * (long long)sizeof(T)) % 16 == 0;
  auto kern = vec ? dequantize_kernel<T, BLOCK, true> : dequantize_kernel<T, BLOCK, false>;
  return launch_chained(kern, grid, 256, 0, 1, s, in, rows, cols, static_cast<T*>(y));
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
  if (by_clusters(a, block))
    *kernel_name = a.out_rows ? "fp4_quantize_rows+fp4_quantize_columns_cluster" : "fp4_quantize_columns_cluster";
  else
    *kernel_name = a.out_rows ? (block == 16 ? "fp4_absmax+fp4_quantize_both" : "fp4_quantize_both")
                              : (block == 16 ? "fp4_absmax+fp4_quantize_columns" : "fp4_quantize_columns");
  if (bf16) return block == 16 ? launch_tiles<__nv_bfloat16, 16>(a, s) : launch_tiles<__nv_bfloat16, 32>(a, s);
  return block == 16 ? launch_tiles<float, 16>(a, s) : launch_tiles<float, 32>(a, s);
}

cudaError_t launch_fp4_dequantize(const void* packed, long long rows, long long cols, int block, void* y, bool bf16,
                                  cudaStream_t s, const char** kernel_name) {
  using namespace fp4;
  *kernel_name = "fp4_dequantize";
  const uint8_t* in = static_cast<const uint8_t*>(packed);
  if (bf16)
    return block == 16 ? launch_dequantize<__nv_bfloat16, 16>(in, rows, cols, y, s)
                       : launch_dequantize<__nv_bfloat16, 32>(in, rows, cols, y, s);
  return block == 16 ? launch_dequantize<float, 16>(in, rows, cols, y, s)
                     : launch_dequantize<float, 32>(in, rows, cols, y, s);
}

}  // namespace qmm
