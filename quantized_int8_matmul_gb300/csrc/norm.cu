// Root-mean-square norm with the residual's addition and an int8 output with
// one scale per row (the A and act_scale of qmm_a8w8), its gradient, and the
// int8 rows read back.
//
// Forward, one row: h = T(x + residual); v = h * w; a = max |v|;
//   rstd = 1 / sqrt(mean(h^2) + eps);  q = rne(v * (127 / a));  scale = a * rstd / 127.
// The normalised row is v * rstd and its largest magnitude a * rstd, so rstd
// cancels out of q: the integers depend on v and its maximum alone (each step
// one rounding, no sum in it), and the row's two reductions (the sum of
// squares, the maximum) run side by side in one pass.
// Backward, one row, the quantiser passed straight through: n = h * rstd,
//   g = dy * w;  dx = rstd * (g - n * mean(g * n)) (+ dh);  dw = sum over rows of dy * n.
// Sums and statistics are fp32 (rows whose squares leave its range: rescaled_row). Both
// are bound by HBM: every tensor is read or written once, the row held in registers
// between its reduction and its output (rows too long for that are read twice).
#include "chain.cuh"
#include "common.cuh"
#include "kernels.h"
#include "row_copy.h"

#include <algorithm>
#include <mutex>

namespace qmm {
namespace norm {

constexpr unsigned kInfBits = 0x7f800000u;

template <typename T>
struct Vec;   // 16 bytes of T
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T>
__device__ __forceinline__ T from_f(float v);   // rounded to nearest even
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The elements a thread holds, NV vectors of E; where vector j of thread t of a row
// of G threads lies (W):
//   kAligned   elements (j * G + t) * E + e, one 16-byte access: every row starts
//              on 16 bytes and holds whole vectors
//   kShifted   the same s elements earlier, s the row's start past a 16-byte
//              boundary: the vectors are aligned, the first and the last of a row
//              are taken element by element (widths that are no multiple of 16
//              bytes: all tensors of a row then start equally far past one)
//   kScalar    (j * E + e) * G + t, element by element (neighbouring threads,
//              neighbouring elements): tensors aligned unlike each other
//   kExact     kAligned where the threads' vectors are the row exactly and the
//              weight has the rows' type: no bound is checked
enum Access { kScalar, kAligned, kShifted, kExact };
template <typename T, int W>
__device__ __forceinline__ int elem(int j, int e, int t, int G, int s) {
  constexpr int E = Vec<T>::E;
  return W == kScalar ? (j * E + e) * G + t : (j * G + t) * E + e - (W == kShifted ? s : 0);
}
template <typename T, int W>
__device__ __forceinline__ int row_shift(long long m, int n) {
  return W == kShifted ? (int)((m * n) & (Vec<T>::E - 1)) : 0;
}
// Vector j is one access (which may lie past the end of the row).
template <typename T, int W>
__device__ __forceinline__ bool whole(int i, int n) {
  return W == kAligned || W == kExact || (W == kShifted && i >= 0 && i + Vec<T>::E <= n);
}
// Vector j of a row of n elements, as 16 bytes of T; elements past the end are 0.
template <typename T, int W>
__device__ __forceinline__ uint4 load_vec(const T* row, int j, int t, int G, int s, int n) {
  constexpr int E = Vec<T>::E;
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  const int i0 = elem<T, W>(j, 0, t, G, s);
  if (whole<T, W>(i0, n)) {
    if (W == kExact || i0 < n) r = *reinterpret_cast<const uint4*>(row + i0);
  } else if (W == kScalar || i0 < n) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = elem<T, W>(j, e, t, G, s);
      if (W == kShifted && i < 0) continue;
      if (sizeof(T) == 4) {
        if (i < n) w[e & 3] = reinterpret_cast<const uint32_t*>(row)[i];
      } else if (i < n) {
        w[(e >> 1) & 3] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << (16 * (e & 1));
      }
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}
template <typename T, int W>
__device__ __forceinline__ void store_vec(T* row, int j, int t, int G, int s, int n, const uint4& r) {
  constexpr int E = Vec<T>::E;
  const int i0 = elem<T, W>(j, 0, t, G, s);
  if (whole<T, W>(i0, n)) {
    if (W == kExact || i0 < n) *reinterpret_cast<uint4*>(row + i0) = r;
  } else if (W == kScalar || i0 < n) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = elem<T, W>(j, e, t, G, s);
      if (i >= n || i < 0) continue;
      if (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row)[i] = w[e & 3];
      else reinterpret_cast<uint16_t*>(row)[i] = (uint16_t)(w[(e >> 1) & 3] >> (16 * (e & 1)));
    }
  }
}
// x + residual rounded to T, element by element.
template <typename T>
__device__ __forceinline__ uint4 add_vec(const uint4& x, const uint4& r) {
  constexpr int E = Vec<T>::E;
  float a[E], b[E];
  Vec<T>::unpack(x, a);
  Vec<T>::unpack(r, b);
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = __fadd_rn(a[e], b[e]);
  return Vec<T>::pack(a);
}
// The E elements that start s before vector v of a 16-byte aligned array (s the
// same for the whole warp; v > 0 unless s is 0), from the two vectors they lie in.
template <typename T>
__device__ __forceinline__ uint4 load_back(const void* base, int v, int s) {
  const uint4* p = static_cast<const uint4*>(base) + v;
  const uint4 b = __ldg(p);
  if (s == 0) return b;
  const uint4 a = __ldg(p - 1);
  uint32_t c[5];
  switch (sizeof(T) == 4 ? s : (s + 1) >> 1) {   // words that a gives
    case 1: c[0] = a.w, c[1] = b.x, c[2] = b.y, c[3] = b.z, c[4] = b.w; break;
    case 2: c[0] = a.z, c[1] = a.w, c[2] = b.x, c[3] = b.y, c[4] = b.z; break;
    case 3: c[0] = a.y, c[1] = a.z, c[2] = a.w, c[3] = b.x, c[4] = b.y; break;
    default: c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = b.x; break;
  }
  if (sizeof(T) == 2 && (s & 1)) {
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = c[k] >> 16 | c[k + 1] << 16;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}
// The weight's elements at the same places (either type; kAligned: 16-byte aligned).
template <typename T, int W>
__device__ __forceinline__ void load_w(const void* w, int w_f32, int j, int t, int G, int s, int n, float* v) {
  constexpr int E = Vec<T>::E;
  if (W == kExact) {
    Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w) + elem<T, W>(j, 0, t, G, s))), v);
  } else if (W == kAligned) {
    const int i = elem<T, W>(j, 0, t, G, s);
    if (i >= n) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
    } else if (w_f32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + i);
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const float4 f = __ldg(p + q);
        v[4 * q] = f.x;
        v[4 * q + 1] = f.y;
        v[4 * q + 2] = f.z;
        v[4 * q + 3] = f.w;
      }
    } else {
      uint32_t f[4];
      if (E == 8) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + i));
        f[0] = r.x;
        f[1] = r.y;
        f[2] = r.z;
        f[3] = r.w;
      } else {
        const uint2 r = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + i));
        f[0] = r.x;
        f[1] = r.y;
      }
#pragma unroll
      for (int q = 0; q < E / 2; ++q) {
        v[2 * q] = __uint_as_float(f[q] << 16);
        v[2 * q + 1] = __uint_as_float(f[q] & 0xffff0000u);
      }
    }
  } else {
    const int i0 = elem<T, W>(j, 0, t, G, s);
    if (W == kShifted && i0 >= 0 && i0 + s + E <= n && (w_f32 != 0) == (sizeof(T) == 4) &&
        (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
      Vec<T>::unpack(load_back<T>(w, (i0 + s) / E, s), v);
      return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = elem<T, W>(j, e, t, G, s);
      v[e] = i >= n || i < 0 ? 0.f
             : w_f32 ? __ldg(static_cast<const float*>(w) + i)
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
    }
  }
}

// Sum of a and maximum of b over the threads of a row: a warp, or the CTA
// through sa / sb (one entry a warp). One barrier: two calls in a row use
// different arrays.
__device__ __forceinline__ void row_sum_max(float& a, unsigned& b, int G, float* sa, unsigned* sb) {
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  b = __reduce_max_sync(0xffffffffu, b);
  if (G == 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = G >> 5;
  if (lane == 0) {
    sa[warp] = a;
    sb[warp] = b;
  }
  __syncthreads();
  a = lane < nw ? sa[lane] : 0.f;
  b = lane < nw ? sb[lane] : 0u;
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  b = __reduce_max_sync(0xffffffffu, b);
}
__device__ __forceinline__ float row_sum(float a, int G, float* sa) {
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (G == 32) return a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = G >> 5;
  if (lane == 0) sa[warp] = a;
  __syncthreads();
  a = lane < nw ? sa[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// The row's scale and the multiplier of v. A row whose v holds a NaN or an
// infinity gets a NaN scale (and zeros); a row with a below 2^-100 (whose 127 / a
// could overflow) is stored as zeros, scale 1.
struct RowScale {
  float inv, scale, rstd;
};
__device__ __forceinline__ RowScale row_scale(float ss, unsigned amax_bits, int n, float eps) {
  RowScale r;
  const float a = __uint_as_float(amax_bits);
  r.rstd = rsqrtf(__fadd_rn(__fdiv_rn(ss, (float)n), eps));
  r.inv = 0.f;
  r.scale = 1.f;
  if (amax_bits >= kInfBits) {
    r.scale = __uint_as_float(0x7fffffffu);
  } else if (a >= 0x1p-100f) {
    r.inv = __fdiv_rn(127.f, a);
    r.scale = __fmul_rn(__fmul_rn(a, r.rstd), 1.f / 127.f);
  }
  return r;
}
// The power of two that brings a row's h into range where the sum of its squares has
// left float32's (1: it has not), the same for all threads of the row.
//   ss infinite: |h| up to 2^128; times 2^-80 the sum of 2^31 squares is below 2^127,
//     and the largest |h|, above 2^48, keeps a square above 2^-64.
//   ss below 2^-90: squares may have lost bits below 2^-126 (a mean wrong by up to
//     2^-149), which shows unless eps covers it: 2^-120 does. Times 2^100 the sum is
//     below 2^110, the smallest |h|, 2^-149, has a square of 2^-98, and eps * 2^200 is
//     below 2^80.
__device__ __forceinline__ float rescale(float ss, float eps) {
  if (__float_as_uint(ss) == kInfBits) return 0x1p-80f;
  return ss < 0x1p-90f && eps < 0x1p-120f ? 0x1p100f : 1.f;
}
// Two float32 operations in one instruction, each rounded once.
__device__ __forceinline__ void mul_pair(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
__device__ __forceinline__ void add_pair(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// (a, b) += (x * z, y * w)
__device__ __forceinline__ void fma_pair(float& a, float& b, float x, float y, float z, float w) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%0, %1};\n\t"
      "fma.rn.f32x2 r, p, q, r;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y), "f"(z), "f"(w));
}
// (c, d) += (a * a, b * b)
__device__ __forceinline__ void square_pair(float a, float b, float& c, float& d) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%0, %1};\n\tfma.rn.f32x2 q, p, p, q;\n\t"
      "mov.b64 {%0, %1}, q;\n\t}"
      : "+f"(c), "+f"(d)
      : "f"(a), "f"(b));
}

// E quantised values as bytes, the first in the lowest. |v * inv| is at most
// 127 (1 + 2^-23), and adding 1.5 * 2^23 rounds such a value to the nearest
// integer (ties to even) and leaves it in the low bits of the sum: one addition
// where a conversion runs at an eighth of its rate.
template <int E>
__device__ __forceinline__ void quantise(const float* v, float inv, bool zero, uint32_t (&o)[E / 4]) {
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    float b[4];
    uint32_t i[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = v[4 * q + e];
#pragma unroll
    for (int e = 0; e < 4; e += 2) mul_pair(b[e], b[e + 1], inv, inv);
    // (one by one: paired, the addition would be fused with the product, whose own
    // rounding the definition has)
#pragma unroll
    for (int e = 0; e < 4; ++e) i[e] = __float_as_uint(__fadd_rn(b[e], 12582912.f));
    o[q] = zero ? 0u : prmt(prmt(i[0], i[1], 0x0040u), prmt(i[2], i[3], 0x0040u), 0x5410u);
  }
}
// max(a, |b|) that keeps a NaN
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// rstd and the scale, once more, of a row whose squares have left float32's range: the
// sum of (f * h)^2, the row of h (a stored one, which may lie over x or the residual,
// else T(x + residual)) read again element by element, and f undone in both. Its int8
// values are right as they are (no sum is in them), so this comes last, when the row's
// registers are free, as a call of its own with the kernel's arguments one by one: ahead
// of the int8 values it held 12 registers more of every row's threads, inlined it cost
// rows that never come here up to 5 % (so 1 %). What the row's threads stored of h is
// visible to all of them: a barrier lies between.
template <typename T>
__device__ __noinline__ void rescaled_row(const void* x, long long ldx, const void* residual, long long ldr,
                                          const void* stored, int n, float eps, float* scale, float* rstd, float* sa,
                                          unsigned amax_bits, float f) {
  const int G = blockDim.x, t = threadIdx.x;
  const long long m = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const T* h = stored ? static_cast<const T*>(stored) + m * n : static_cast<const T*>(x) + m * ldx;
  const T* r = residual && !stored ? static_cast<const T*>(residual) + m * ldr : nullptr;
  if (G == 32) __syncwarp();
  float ss = 0.f;
#pragma unroll 1
  for (int i = t; i < n; i += G) {
    float a = (float)h[i];
    if (r) a = (float)from_f<T>(__fadd_rn(a, (float)r[i]));
    a = __fmul_rn(a, f);
    ss = __fmaf_rn(a, a, ss);
  }
  if (G > 32) __syncthreads();   // sa has been read
  ss = row_sum(ss, G, sa);
  if (t != 0) return;
  const float root = rsqrtf(__fadd_rn(__fdiv_rn(ss, (float)n), __fmul_rn(__fmul_rn(eps, f), f)));
  if (rstd) rstd[m] = __fmul_rn(f, root);
  const float a = __uint_as_float(amax_bits);
  if (amax_bits < kInfBits && a >= 0x1p-100f) scale[m] = __fmul_rn(__fmul_rn(__fmul_rn(a, f), root), 1.f / 127.f);
}

// One row per G = blockDim.x threads (blockDim.y rows a CTA where G is a warp),
// NV vectors a thread. NV = 0: rows of any length, read twice.
// 8192 x 4096 bf16: 36.1 us with a residual (6.5 TB/s, 97 % of a copy's rate), 19.0
// without (5.3 TB/s: then a CTA's two barriers a row show); 4096 x 11008 float32
// with one 103 us (85 %). Rows that start off 16 bytes: 8192 x 4095 bf16 57 us,
// 1009 x 5003 float32 9.1 us (2.8 TB/s; the weight comes by two vectors and a shift,
// 9.6 us element by element; a row's first and last vectors go element by element).
template <typename T, int W, int NV>
__global__ void __launch_bounds__(1024) rms_norm_s8_kernel(const NormArgs p) {
  constexpr int E = Vec<T>::E;
  __shared__ float sa[32];
  __shared__ unsigned sb[32];
  chain_wait();
  const int n = p.H, G = blockDim.x, t = threadIdx.x;
  const long long m = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (m >= p.M) return;   // whole warps (G a warp), or nobody
  const int s = row_shift<T, W>(m, n);
  const T* x = static_cast<const T*>(p.x) + m * p.ldx;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + m * p.ldr : nullptr;
  T* ho = p.h ? static_cast<T*>(p.h) + m * (long long)n : nullptr;
  int8_t* q = p.q + m * (long long)n;
  float ss = 0.f, ss2 = 0.f, amax = 0.f;   // the even and the odd elements' squares
  // v = h * w of a vector, and its share of the statistics
  auto stats = [&](const uint4& hr, const float* w, float* v) {
    Vec<T>::unpack(hr, v);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      square_pair(v[e], v[e + 1], ss, ss2);
      mul_pair(v[e], v[e + 1], w[e], w[e + 1]);
      amax = max_abs(max_abs(amax, v[e]), v[e + 1]);
    }
  };
  auto rescaled = [&](unsigned am) {
    const float f = rescale(ss, p.eps);
    if (__builtin_expect(f != 1.f, 0))
      rescaled_row<T>(p.x, p.ldx, p.residual, p.ldr, p.h, n, p.eps, p.scale, p.rstd, sa, am, f);
  };
  auto put = [&](int j, const float* v, float inv, bool zero) {
    uint32_t o[E / 4];
    quantise<E>(v, inv, zero, o);
    const int i0 = elem<T, W>(j, 0, t, G, s);
    if (whole<T, W>(i0, n)) {
      if (W != kExact && i0 >= n) return;
      if (E == 8) *reinterpret_cast<uint2*>(q + i0) = make_uint2(o[0], o[E / 4 - 1]);
      else *reinterpret_cast<uint32_t*>(q + i0) = o[0];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = elem<T, W>(j, e, t, G, s);
        if (i < n && i >= 0) q[i] = (int8_t)(o[e >> 2] >> (8 * (e & 3)));
      }
    }
  };
  if (NV > 0) {
    constexpr int K = NV > 0 ? NV : 1;
    uint4 h[K];
    float v[K][E];
#pragma unroll
    for (int j = 0; j < K; ++j) h[j] = load_vec<T, W>(x, j, t, G, s, n);
    if (r) {
      uint4 b[K];
#pragma unroll
      for (int j = 0; j < K; ++j) b[j] = load_vec<T, W>(r, j, t, G, s, n);
#pragma unroll
      for (int j = 0; j < K; ++j) h[j] = add_vec<T>(h[j], b[j]);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (ho) store_vec<T, W>(ho, j, t, G, s, n, h[j]);
      float w[E];
      load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
      stats(h[j], w, v[j]);
    }
    unsigned am = __float_as_uint(amax);
    ss += ss2;
    row_sum_max(ss, am, G, sa, sb);
    const RowScale rs = row_scale(ss, am, n, p.eps);
    chain_release();
    if (t == 0) {
      p.scale[m] = rs.scale;
      if (p.rstd) p.rstd[m] = rs.rstd;
    }
#pragma unroll
    for (int j = 0; j < K; ++j) put(j, v[j], rs.inv, am >= kInfBits);
    rescaled(am);
  } else {
    const int steps = (n + s + G * E - 1) / (G * E);
    for (int j = 0; j < steps; ++j) {
      uint4 h = load_vec<T, W>(x, j, t, G, s, n);
      if (r) h = add_vec<T>(h, load_vec<T, W>(r, j, t, G, s, n));
      if (ho) store_vec<T, W>(ho, j, t, G, s, n, h);
      float v[E], w[E];
      load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
      stats(h, w, v);
    }
    unsigned am = __float_as_uint(amax);
    ss += ss2;
    row_sum_max(ss, am, G, sa, sb);
    const RowScale rs = row_scale(ss, am, n, p.eps);
    chain_release();
    if (t == 0) {
      p.scale[m] = rs.scale;
      if (p.rstd) p.rstd[m] = rs.rstd;
    }
    for (int j = 0; j < steps; ++j) {
      // a stored h is read back (by the thread that wrote it: it may lie over x or the residual)
      uint4 h = load_vec<T, W>(ho ? ho : x, j, t, G, s, n);
      if (r && !ho) h = add_vec<T>(h, load_vec<T, W>(r, j, t, G, s, n));
      float v[E], w[E];
      load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
      Vec<T>::unpack(h, v);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = __fmul_rn(v[e], w[e]);
      put(j, v, rs.inv, am >= kInfBits);
    }
    rescaled(am);
  }
}

// y[i] = q[i] * scale[i / H] over the flat [M * H] array, eight elements a step
// (both arrays are contiguous, so no width is unaligned). 8192 x 4096 to bf16: 16.3
// us, 6.2 TB/s, 92 % of a copy's rate; 4096 x 11008 to float32 33.9 us, 99 % (42.8
// with a lane's 32 bytes in two stores).
template <typename T, typename I, bool VEC>
__global__ void __launch_bounds__(256) s8_dequantize_rows_kernel(const int8_t* q, const float* scale, I total, I H,
                                                                 T* y) {
  chain_wait();
  constexpr int STEPS = 2;
  uint2 raw[STEPS];
  const I base = (I)blockIdx.x * (256 * 8 * STEPS) + threadIdx.x * 8;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const I i = base + (I)s * (256 * 8);
    if (VEC && i < total && total - i >= 8) raw[s] = *reinterpret_cast<const uint2*>(q + i);
  }
  chain_release();
  const bool wide = (reinterpret_cast<uintptr_t>(y) & 31) == 0;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const I i = base + (I)s * (256 * 8);
    if (i >= total) return;
    const I m = i / H, c = i - m * H;
    if (VEC && total - i >= 8) {
      float f[8];
      const uint32_t w[2] = {raw[s].x, raw[s].y};
      const float s0 = __ldg(scale + m);
      if (H - c >= 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fmul_rn((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))), s0);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          f[e] = __fmul_rn((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))), __ldg(scale + (i + e) / H));
      }
      if (sizeof(T) == 4 && wide) {   // a whole 32-byte sector a lane
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y + i), "f"(f[0]), "f"(f[1]),
                     "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += Vec<T>::E) *reinterpret_cast<uint4*>(y + i + e) = Vec<T>::pack(f + e);
      }
    } else {
      for (int e = 0; e < 8 && total - i > (I)e; ++e)
        y[i + e] = from_f<T>(__fmul_rn((float)q[i + e], __ldg(scale + (i + e) / H)));
    }
  }
}

// Backward. A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ... (blockDim.y
// of them at a time where a row is one warp's) and keeps its columns' share of
// dweight in registers; the shares go to partials and sum_partials adds them in
// order. This one loads rows directly: rows of one warp, tensors aligned unlike
// each other, and (NV = 0) rows too long for registers, which are read twice, the
// shares of dweight accumulated in partials itself. Bound by the latency of a row's
// loads, reduction and stores: 8192 x 256 bf16 8.2 us (2.0 TB/s).
template <typename T, int W, int NV, bool DH>
__global__ void __launch_bounds__(1024)
    rms_norm_backward_kernel(const NormBwdArgs p) {
  constexpr int E = Vec<T>::E;
  constexpr int K = NV > 0 ? NV : 1;
  __shared__ float sa[2][32];
  __shared__ float sw[NV == 1 ? 8 * 32 * E : 1];
  chain_wait();
  const int n = p.H, G = blockDim.x, t = threadIdx.x;
  const long long step = (long long)gridDim.x * blockDim.y;
  const T* h0 = static_cast<const T*>(p.h);
  const T* dy0 = static_cast<const T*>(p.dy);
  const T* dh0 = DH ? static_cast<const T*>(p.dh) : nullptr;
  float* part = p.partials + (long long)blockIdx.x * n;
  long long m = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  // the same for all rows of a thread: their distance is a multiple of E rows (or
  // there is one row), so its columns stay the same
  const int s = row_shift<T, W>(m, n);
  int par = 0;
  if (NV > 0) {
    constexpr bool HELD = NV == 1;   // the weight in registers too
    float dw[K][E], w[E];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) dw[j][e] = 0.f;
    if (HELD) load_w<T, W>(p.w, p.w_f32, 0, t, G, s, n, w);
    for (; m < p.M; m += step) {
      const float rstd = __ldg(p.rstd + m);
      uint4 h[K], dy[K], dh[DH ? K : 1];
#pragma unroll
      for (int j = 0; j < K; ++j) h[j] = load_vec<T, W>(h0 + m * p.ldh, j, t, G, s, n);
#pragma unroll
      for (int j = 0; j < K; ++j) dy[j] = load_vec<T, W>(dy0 + m * p.lddy, j, t, G, s, n);
      if (DH) {
#pragma unroll
        for (int j = 0; j < K; ++j) dh[DH ? j : 0] = load_vec<T, W>(dh0 + m * p.lddh, j, t, G, s, n);
      }
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float nn[E], g[E];
        if (!HELD) load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
        Vec<T>::unpack(h[j], nn);
        Vec<T>::unpack(dy[j], g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          nn[e] *= rstd;
          dw[j][e] = __fmaf_rn(g[e], nn[e], dw[j][e]);
          dot = __fmaf_rn(g[e] * w[e], nn[e], dot);
        }
      }
      const float c = -(row_sum(dot, G, sa[par]) / (float)n) * rstd;   // dx = g * rstd + n * c
      par ^= 1;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float v[E], g[E];
        if (!HELD) load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
        Vec<T>::unpack(h[j], v);
        Vec<T>::unpack(dy[j], g);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(v[e] * rstd, c, g[e] * w[e] * rstd);
        if (DH) {
          Vec<T>::unpack(dh[DH ? j : 0], g);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += g[e];
        }
        store_vec<T, W>(static_cast<T*>(p.dx) + m * (long long)n, j, t, G, s, n, Vec<T>::pack(v));
      }
    }
    chain_release();
    if (NV == 1 && blockDim.y > 1) {   // the CTA's warps, each with rows of its own: added in order
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = elem<T, W>(0, e, t, G, s);
        if (i >= 0 && i < n) sw[threadIdx.y * 32 * E + i] = dw[0][e];
      }
      __syncthreads();
      for (int i = threadIdx.y * 32 + t; i < n; i += 32 * blockDim.y) {
        float a = sw[i];
        for (int y = 1; y < (int)blockDim.y; ++y) a += sw[y * 32 * E + i];
        part[i] = a;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = elem<T, W>(j, e, t, G, s);
        if (i < n && i >= 0) part[i] = dw[j][e];
      }
  } else {
    const int steps = (n + s + G * E - 1) / (G * E);
    bool fresh = true;
    for (; m < p.M; m += step) {
      const float rstd = __ldg(p.rstd + m);
      float dot = 0.f;
      for (int j = 0; j < steps; ++j) {
        float h[E], dy[E], w[E];
        Vec<T>::unpack(load_vec<T, W>(h0 + m * p.ldh, j, t, G, s, n), h);
        Vec<T>::unpack(load_vec<T, W>(dy0 + m * p.lddy, j, t, G, s, n), dy);
        load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
#pragma unroll
        for (int e = 0; e < E; ++e) dot = __fmaf_rn(dy[e] * w[e], h[e] * rstd, dot);
      }
      const float mean = row_sum(dot, G, sa[par]) / (float)n;
      par ^= 1;
      for (int j = 0; j < steps; ++j) {
        float h[E], dy[E], dh[E], w[E];
        Vec<T>::unpack(load_vec<T, W>(h0 + m * p.ldh, j, t, G, s, n), h);
        Vec<T>::unpack(load_vec<T, W>(dy0 + m * p.lddy, j, t, G, s, n), dy);
        if (DH) Vec<T>::unpack(load_vec<T, W>(dh0 + m * p.lddh, j, t, G, s, n), dh);
        load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float nn = h[e] * rstd;
          const int i = elem<T, W>(j, e, t, G, s);
          if (i < n && i >= 0) part[i] = __fmaf_rn(dy[e], nn, fresh ? 0.f : part[i]);
          h[e] = __fmaf_rn(-nn, mean, dy[e] * w[e]) * rstd;
          if (DH) h[e] += dh[e];
        }
        store_vec<T, W>(static_cast<T*>(p.dx) + m * (long long)n, j, t, G, s, n, Vec<T>::pack(h));
      }
      fresh = false;
    }
  }
}

// The same for rows that come by bulk copies: a ring of `slots` rows (h, dy and dh
// each in 16-byte lines; of rows too long for two slots of all three, h and dy) in
// shared memory, refilled once a row's reduction has passed, so that the next rows
// are on their way through the whole of this one's work. No copy reaches past the last
// row of a tensor (4096 x 4095 bf16 with dh 49.1 us; 47.2 if the last one might). Rows of one vector a
// thread go in pairs (RB = 2): one barrier and one reduction for both (8192 x 1024
// bf16 21.1 -> 19.8 us). With sum_partials: 4096 x 4096 bf16 with dh 30.1 us (4.5
// TB/s, 67 %), 4096 x 8192 49.9 (80 %), 1531 x 11008 float32 43.5 (69 %; 1531 rows
// on 152 CTAs are eleven rounds for the longest and ten for the others). Of the 30.1
// the ring takes 26, the rest is the partial sums' own launch and pass. Waits are
// bounded (common.cuh).
constexpr int RING_MAX = 8;
constexpr unsigned SITE_ROW = 0x520;

// sums of RB values over the CTA's threads; sa: [RB][32]
template <int RB>
__device__ __forceinline__ void row_sums(float (&a)[RB], int G, float* sa) {
  if constexpr (RB == 1) {
    a[0] = row_sum(a[0], G, sa);
  } else {   // the halves of a warp take a row each
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = G >> 5, hi = lane >> 4, l = lane & 15;
    float v = (hi ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, hi ? a[0] : a[1], 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (G > 32) {
      if (l == 0) sa[hi * 32 + warp] = v;
      __syncthreads();
      v = (l < nw ? sa[hi * 32 + l] : 0.f) + (l + 16 < nw ? sa[hi * 32 + l + 16] : 0.f);
#pragma unroll
      for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    a[0] = __shfl_sync(0xffffffffu, v, 0);
    a[1] = __shfl_sync(0xffffffffu, v, 16);
  }
}

template <typename T, int W, int NV, bool DH, int RB>
__global__ void __launch_bounds__(1024) rms_norm_backward_ring_kernel(const NormBwdArgs p, const int slots,
                                                                      const int tensors) {
  constexpr int E = Vec<T>::E;
  constexpr bool HELD = NV == 1;   // the weight in registers too
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float sa[2][RB * 32];
  __shared__ uint64_t full[RING_MAX];
  chain_wait();
  const int n = p.H, G = blockDim.x, t = threadIdx.x;
  const long long m0 = blockIdx.x, step = gridDim.x;
  const int rows = (int)((p.M - m0 + step - 1) / step);
  const int s = row_shift<T, W>(m0, n);   // the same for all of the CTA's rows
  const uint32_t pitch = (uint32_t)(n + E) * (uint32_t)sizeof(T) / 16u * 16u + 16u;
  // The end of the tensors' last row is not copied (row_copy.h). The CTA that has the row
  // reads it element by element: into the row's slot where that is filled at the start,
  // else into its own row of partials, which it needs at its end only, from where a copy
  // takes it to the slot behind the row before it.
  auto tails = [&] {   // 16 bytes a tensor
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p.partials + m0 * n) + 15) & ~(uintptr_t)15);
  };
  auto fill = [&](int r) {   // one thread
    const long long m = m0 + r * step;
    uint64_t* bar = &full[r % slots];
    const uint32_t dst = smem_u32(ring) + (uint32_t)(r % slots) * (uint32_t)tensors * pitch;
    const bool last = W == kShifted && m == p.M - 1;
    const uint32_t bytes = row_copy_bytes(n, s, (int)sizeof(T), last);
    const uint32_t end = last && r >= slots ? row_copy_bytes(n, s, (int)sizeof(T), false) - bytes : 0u;   // 0 or 16
    mbar_arrive_expect_tx(bar, (uint32_t)tensors * (bytes + end));
    if (end)
#pragma unroll 1
      for (int i = 0; i < tensors; ++i) bulk_load(dst + i * pitch + bytes, tails() + 16 * i, end, bar);
    bulk_load(dst, static_cast<const T*>(p.h) + m * p.ldh - s, bytes, bar);
    bulk_load(dst + pitch, static_cast<const T*>(p.dy) + m * p.lddy - s, bytes, bar);
    if (DH && tensors == 3) bulk_load(dst + 2 * pitch, static_cast<const T*>(p.dh) + m * p.lddh - s, bytes, bar);
  };
  if (t == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
    for (int r = 0; r < slots && r < rows; ++r) fill(r);
  }
  if (W == kShifted && m0 + (rows - 1) * step == p.M - 1) {
    const int last = rows - 1;
    const uint32_t last_line = row_copy_bytes(n, s, (int)sizeof(T), true);
    const int left = (n + s) & (E - 1), which = t / E, k = t & (E - 1);
    if (which < tensors && k < left) {
      const T* end = static_cast<const T*>(which == 0 ? p.h : which == 1 ? p.dy : p.dh) +
                     (p.M - 1) * (which == 0 ? p.ldh : which == 1 ? p.lddy : p.lddh) + n - left;
      uint8_t* to = last < slots ? ring + ((size_t)last * (uint32_t)tensors + which) * pitch + last_line
                                 : tails() + 16 * which;
      reinterpret_cast<T*>(to)[k] = end[k];
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");   // for the copy engine (then the barrier)
  }
  float dw[NV][E], w[E];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[j][e] = 0.f;
  if (HELD) load_w<T, W>(p.w, p.w_f32, 0, t, G, s, n, w);
  __syncthreads();
  // vector j of a row in the ring, with zeros outside the row
  auto get = [&](const uint8_t* row, int j) {
    const int i0 = elem<T, W>(j, 0, t, G, s);
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (W == kExact || i0 < n) r = *reinterpret_cast<const uint4*>(row + (size_t)(j * G + t) * 16);
    if (W == kShifted && i0 < n && !whole<T, W>(i0, n)) {
      float f[E];
      Vec<T>::unpack(r, f);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (i0 + e < 0 || i0 + e >= n) f[e] = 0.f;
      r = Vec<T>::pack(f);
    }
    return r;
  };
  float next[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) next[b] = b < rows ? __ldg(p.rstd + m0 + b * step) : 0.f;
  int slot = 0, seen = 0, got = 0;   // the next row's slot, how often the ring went round, rows that came
  for (int r = 0; r < rows; r += RB) {
    const long long m = m0 + r * step;
    float rstd[RB], dot[RB];
    uint4 h[RB][NV], dy[RB][NV], dh[RB][DH ? NV : 1];
    bool ok = true;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      rstd[b] = next[b];
      next[b] = r + RB + b < rows ? __ldg(p.rstd + m + (RB + b) * step) : 0.f;
      dot[b] = 0.f;
      if (b > 0 && r + b >= rows) {   // a row of zeros (rstd 0)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          h[b][j] = dy[b][j] = make_uint4(0u, 0u, 0u, 0u);
          if (DH) dh[b][j] = h[b][j];
        }
        continue;
      }
      ok = ok && mbar_wait(&full[slot], (uint32_t)(seen & 1), nullptr, p.err, SITE_ROW);
      if (!ok) break;
      const uint8_t* in = ring + (size_t)slot * (uint32_t)tensors * pitch;
      if (++slot == slots) slot = 0, ++seen;
      ++got;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        h[b][j] = get(in, j);
        dy[b][j] = get(in + pitch, j);
        if (DH && tensors == 3) dh[b][DH ? j : 0] = get(in + 2 * pitch, j);
        if (DH && tensors == 2)   // not in the ring: too long
          dh[b][DH ? j : 0] = load_vec<T, W>(static_cast<const T*>(p.dh) + (m + b * step) * p.lddh, j, t, G, s, n);
        float nn[E], g[E], d2[2] = {0.f, 0.f};
        if (!HELD) load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
        Vec<T>::unpack(h[b][j], nn);
        Vec<T>::unpack(dy[b][j], g);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          mul_pair(nn[e], nn[e + 1], rstd[b], rstd[b]);
          fma_pair(dw[j][e], dw[j][e + 1], g[e], g[e + 1], nn[e], nn[e + 1]);
          mul_pair(g[e], g[e + 1], w[e], w[e + 1]);
          fma_pair(d2[0], d2[1], g[e], g[e + 1], nn[e], nn[e + 1]);
        }
        dot[b] += d2[0] + d2[1];
      }
    }
    if (!ok) {   // the copies of the later slots are waited for, with the same limit, before the CTA ends
      for (++got; got < rows && got < r + slots; ++got) {
        if (++slot == slots) slot = 0, ++seen;
        mbar_wait(&full[slot], (uint32_t)(seen & 1), nullptr, p.err, SITE_ROW);
      }
      break;
    }
    // past the barrier in row_sums the rows are in registers and their slots free
    row_sums<RB>(dot, G, sa[(r / RB) & 1]);
    if (t == 0 && r + slots < rows) {
      fence_proxy_async_smem();   // the slots were read through the generic proxy
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (r + b + slots < rows) fill(r + b + slots);
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (b > 0 && r + b >= rows) break;
      const float c = -(dot[b] / (float)n) * rstd[b];   // dx = g * rstd + n * c
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[E], g[E], d[E];
        if (!HELD) load_w<T, W>(p.w, p.w_f32, j, t, G, s, n, w);
        Vec<T>::unpack(h[b][j], v);
        Vec<T>::unpack(dy[b][j], g);
        if (DH) Vec<T>::unpack(dh[b][DH ? j : 0], d);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          mul_pair(v[e], v[e + 1], rstd[b], rstd[b]);
          mul_pair(g[e], g[e + 1], w[e], w[e + 1]);
          mul_pair(g[e], g[e + 1], rstd[b], rstd[b]);
          fma_pair(g[e], g[e + 1], v[e], v[e + 1], c, c);
          if (DH) add_pair(g[e], g[e + 1], d[e], d[e + 1]);
        }
        store_vec<T, W>(static_cast<T*>(p.dx) + (m + b * step) * (long long)n, j, t, G, s, n, Vec<T>::pack(g));
      }
    }
  }
  chain_release();
  float* part = p.partials + m0 * n;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = elem<T, W>(j, e, t, G, s);
      if (i < n && i >= 0) part[i] = dw[j][e];
    }
}

// out[i] = the sum of column i of part [count][n], in a fixed order: a cluster for
// 32 columns, each CTA a run of the rows as 32 interleaved ones (twelve loads of
// each in flight), joined in rank order. 304 x 4096 shares: about 4 us, all latency.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* part, int count, int n, int split,
                                                            float* out) {
  __shared__ float s[32][33];
  __shared__ float sum[32];
  chain_wait();
  const int rank = split > 1 ? (int)cluster_ctarank() : 0, c0 = blockIdx.x / split * 32;
  const int beg = (int)((long long)count * rank / split), end = (int)((long long)count * (rank + 1) / split);
  const int i = c0 + threadIdx.x;
  float a = 0.f;
  if (i < n) {
    for (int c = beg + threadIdx.y; c < end; c += 32 * 12) {
      float v[12];
#pragma unroll
      for (int k = 0; k < 12; ++k) v[k] = c + 32 * k < end ? part[(long long)(c + 32 * k) * n + i] : 0.f;
#pragma unroll
      for (int k = 0; k < 12; ++k) a += v[k];
    }
  }
  chain_release();
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  a = s[threadIdx.x][threadIdx.y];   // one column a warp
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (threadIdx.x == 0) sum[threadIdx.y] = a;
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  if (rank == 0 && threadIdx.y == 0 && i < n) {
    float r = sum[threadIdx.x];
    for (int k = 1; k < split; ++k) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(x)
                   : "r"(mapa_shared(smem_u32(&sum[threadIdx.x]), (uint32_t)k)));
      r += x;
    }
    out[i] = r;
  }
  if (split > 1) cluster_sync_all();   // rank 0 has read the others' sums
}

// A tensor of rows ld apart whose row m starts as far past a 16-byte boundary as
// element m * H of an aligned array.
template <typename T>
bool rows_like(const void* p, long long ld, int H) {
  return !p || ((reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld - H) % Vec<T>::E == 0);
}
// Vectors of a row, shifted if it has to be.
template <typename T>
int row_vectors(int H) {
  constexpr int E = Vec<T>::E;
  return H % E == 0 ? H / E : (H + 2 * (E - 1)) / E;
}

int round32(int v) { return (v + 31) / 32 * 32; }

// Vectors a thread and threads a row. With rows enough to fill the GPU, four
// vectors a thread (fewer warps to run the per-row steps); with few rows one (the
// row's latency). Rows of one warp share a CTA. Long rows are read twice, by CTAs
// small enough that several share an SM: held in registers, a row leaves no room
// for the next one's loads (4096 x 11008 float32: 105 us read twice, 144 held).
template <typename T>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  constexpr int E = Vec<T>::E;
  const bool like = rows_like<T>(a.x, a.ldx, a.H) && rows_like<T>(a.residual, a.ldr, a.H) &&
                    rows_like<T>(a.h, a.H, a.H) && (reinterpret_cast<uintptr_t>(a.q) % 8) == 0;
  const Access acc = !like ? kScalar
                     : a.H % E == 0 && (reinterpret_cast<uintptr_t>(a.w) % 16) == 0 ? kAligned : kShifted;
  const int nvec = row_vectors<T>(a.H);
  const bool many = a.M >= 2 * num_sms();
  int nv = many ? (nvec <= 32 ? 1 : nvec <= 128 ? 2 : 4) : (nvec <= 1024 ? 1 : nvec <= 2048 ? 2 : 4);
  if (nvec > (many ? 2048 : 4096)) nv = 0;
  const int G = nv ? std::max(32, round32((nvec + nv - 1) / nv)) : many ? 512 : 1024;
  const int R = G == 32 ? (many ? 8 : 1) : 1;
  const dim3 block(G, R);
  const unsigned grid = (unsigned)((a.M + R - 1) / R);
#define QMM_NORM(V)                                                                                     \
  switch (nv) {                                                                                         \
    case 1: return launch_chained(rms_norm_s8_kernel<T, V, 1>, grid, block, 0, 1, s, a);                \
    case 2: return launch_chained(rms_norm_s8_kernel<T, V, 2>, grid, block, 0, 1, s, a);                \
    case 4: return launch_chained(rms_norm_s8_kernel<T, V, 4>, grid, block, 0, 1, s, a);                \
    default: return launch_chained(rms_norm_s8_kernel<T, V, 0>, grid, block, 0, 1, s, a);               \
  }
  if (acc == kAligned && nv > 0 && nv * G * E == a.H && (a.w_f32 != 0) == (sizeof(T) == 4)) QMM_NORM(kExact)
  if (acc == kAligned) QMM_NORM(kAligned)
  if (acc == kShifted) QMM_NORM(kShifted)
  QMM_NORM(kScalar)
#undef QMM_NORM
}

template <typename T, typename I>
cudaError_t launch_dequantize_i(const int8_t* q, const float* scale, long long M, int H, T* y, cudaStream_t s) {
  const long long total = M * H;
  const unsigned grid = (unsigned)((total + 4095) / 4096);
  const bool vec = (reinterpret_cast<uintptr_t>(q) % 8) == 0 && (reinterpret_cast<uintptr_t>(y) % 16) == 0;
  auto kern = vec ? s8_dequantize_rows_kernel<T, I, true> : s8_dequantize_rows_kernel<T, I, false>;
  return launch_chained(kern, grid, 256, 0, 1, s, q, scale, (I)total, (I)H, y);
}
template <typename T>
cudaError_t launch_dequantize(const int8_t* q, const float* scale, long long M, int H, T* y, cudaStream_t s) {
  return M * H + 8192 < (1ll << 32) ? launch_dequantize_i<T, uint32_t>(q, scale, M, H, y, s)
                                    : launch_dequantize_i<T, uint64_t>(q, scale, M, H, y, s);
}

// Launch shape of the backward pass: vectors a thread, threads a row, rows of a
// CTA at a time, CTAs (= rows of partials), slots of a CTA's ring (0: direct).
// 64 registers hold one vector of each tensor with its weight and sums, or two, or
// three of float32; longer rows are read twice. CTAs are as many as fit at once
// (1024 threads and the rings' two slots or more an SM, at most 8 an SM), no more
// than rows, or a multiple of 8 (row_shift). They are counted for the 152 SMs of a GB300
// and not the device's own, as the size of the workspace has to come out the same on a
// host without one.
struct BwdShape {
  int nv, G, R, parts, slots, tensors;
  size_t slot;   // bytes: a row of each of `tensors`
};
template <typename T>
BwdShape backward_shape(long long M, int H, bool dh, Access acc) {
  constexpr int MOST = sizeof(T) == 4 ? 3 : 2;   // vectors a thread
  constexpr int E = Vec<T>::E;
  BwdShape b;
  const int nvec = row_vectors<T>(H);
  const size_t row = (size_t)(H + E) * sizeof(T) / 16 * 16 + 16, room = 212 * 1024;
  b.tensors = dh && 2 * 3 * row <= room ? 3 : 2;
  b.slot = b.tensors * row;
  b.R = 1;
  b.slots = 0;
  b.nv = std::max(1, (nvec + 1023) / 1024);
  if (b.nv > MOST) b.nv = 0;
  b.G = b.nv ? std::max(32, round32((nvec + b.nv - 1) / b.nv)) : 1024;
  const int fit = (int)std::min<size_t>(64, room / b.slot);
  int per_sm = std::min(8, 1024 / b.G);
  if (acc != kScalar && b.nv > 0 && b.G > 32 && fit >= 2) {
    per_sm = std::min(per_sm, fit / 2);
    b.slots = std::min(RING_MAX, fit / per_sm);
  } else {
    if (acc == kScalar && b.nv == 3) b.nv = 0, b.G = 1024;
    b.R = b.G == 32 ? 8 : 1;
    per_sm = std::max(1, std::min(8, 1024 / (b.G * b.R)));
  }
  b.parts = (int)std::min<long long>((M + b.R - 1) / b.R, 152ll * per_sm);
  return b;
}

// dweight from the partials.
cudaError_t launch_sum(const NormBwdArgs& a, int parts, cudaStream_t s) {
  const int groups = (a.H + 31) / 32;
  int split = 1;   // up to 8, while that leaves every thread a load and every SM at most one CTA
  while (split < 8 && parts >= 64 * split && groups * split * 2 <= num_sms()) split *= 2;
  return launch_chained(sum_partials_kernel, (unsigned)(groups * split), dim3(32, 32), 0, (unsigned)split, s,
                        a.partials, parts, a.H, split, a.dweight);
}

template <typename T, int W, int NV, bool DH, int RB>
cudaError_t launch_ring_nv(const NormBwdArgs& a, const BwdShape& b, int slots, size_t smem, cudaStream_t s) {
  auto kern = rms_norm_backward_ring_kernel<T, W, NV, DH, RB>;
  static std::once_flag once[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
  });
  if (e != cudaSuccess) return e;
  return launch_chained(kern, b.parts, b.G, smem, 1, s, a, slots, b.tensors);
}
template <typename T, int W, bool DH>
cudaError_t launch_ring(const NormBwdArgs& a, const BwdShape& b, cudaStream_t s) {
  const size_t smem = b.slots * b.slot;
  // (pairs of rows leave two slots on their way)
  if (b.nv == 1 && b.slots >= 4) return launch_ring_nv<T, W, 1, DH, 2>(a, b, b.slots, smem, s);
  if (b.nv == 1) return launch_ring_nv<T, W, 1, DH, 1>(a, b, b.slots, smem, s);
  if (b.nv == 2) return launch_ring_nv<T, W, 2, DH, 1>(a, b, b.slots, smem, s);
  return launch_ring_nv<T, W, sizeof(T) == 4 ? 3 : 2, DH, 1>(a, b, b.slots, smem, s);
}

// (of aligned tensors only rows of one warp and rows too long come here)
template <typename T, int W, bool DH>
cudaError_t launch_direct(const NormBwdArgs& a, const BwdShape& b, cudaStream_t s) {
  constexpr int NV2 = W == kScalar ? 2 : 0;
  auto kern = b.nv == 1   ? rms_norm_backward_kernel<T, W, 1, DH>
              : b.nv == 2 ? rms_norm_backward_kernel<T, W, NV2, DH>
                          : rms_norm_backward_kernel<T, W, 0, DH>;
  return launch_chained(kern, b.parts, dim3(b.G, b.R), 0, 1, s, a);
}

template <typename T, bool DH>
cudaError_t launch_backward(const NormBwdArgs& a, cudaStream_t s) {
  constexpr int E = Vec<T>::E;
  const bool like = rows_like<T>(a.h, a.ldh, a.H) && rows_like<T>(a.dy, a.lddy, a.H) &&
                    rows_like<T>(a.dh, a.lddh, a.H) && rows_like<T>(a.dx, a.H, a.H);
  const Access acc = !like ? kScalar
                     : a.H % E == 0 && (reinterpret_cast<uintptr_t>(a.w) % 16) == 0 ? kAligned : kShifted;
  const BwdShape b = backward_shape<T>(a.M, a.H, DH, acc);
  cudaError_t e;
  if (b.slots > 0)
    e = acc == kShifted ? launch_ring<T, kShifted, DH>(a, b, s)
        : b.nv * b.G * E == a.H && (a.w_f32 != 0) == (sizeof(T) == 4) ? launch_ring<T, kExact, DH>(a, b, s)
                                                                       : launch_ring<T, kAligned, DH>(a, b, s);
  else
    e = acc == kAligned   ? launch_direct<T, kAligned, DH>(a, b, s)
        : acc == kShifted ? launch_direct<T, kShifted, DH>(a, b, s)
                          : launch_direct<T, kScalar, DH>(a, b, s);
  return e != cudaSuccess ? e : launch_sum(a, b.parts, s);
}

}  // namespace norm

cudaError_t launch_rms_norm_s8(const NormArgs& a, bool bf16, cudaStream_t s, const char** kernel_name) {
  *kernel_name = "rms_norm_s8";
  return bf16 ? norm::launch_norm<__nv_bfloat16>(a, s) : norm::launch_norm<float>(a, s);
}

cudaError_t launch_s8_dequantize_rows(const int8_t* q, const float* scale, long long M, int H, void* y, bool bf16,
                                      cudaStream_t s, const char** kernel_name) {
  *kernel_name = "s8_dequantize_rows";
  return bf16 ? norm::launch_dequantize(q, scale, M, H, static_cast<__nv_bfloat16*>(y), s)
              : norm::launch_dequantize(q, scale, M, H, static_cast<float*>(y), s);
}

// The largest count over what the size query does not know: type, dh, alignment.
int rms_norm_backward_partials(long long M, int H) {
  int most = 0;
  for (const norm::Access acc : {norm::kScalar, norm::kAligned})
    for (const bool dh : {false, true})
      most = std::max({most, norm::backward_shape<float>(M, H, dh, acc).parts,
                       norm::backward_shape<__nv_bfloat16>(M, H, dh, acc).parts});
  return most;
}

cudaError_t launch_rms_norm_backward(const NormBwdArgs& a, bool bf16, cudaStream_t s, const char** kernel_name) {
  *kernel_name = "rms_norm_backward+sum_partials";
  if (bf16)
    return a.dh ? norm::launch_backward<__nv_bfloat16, true>(a, s) : norm::launch_backward<__nv_bfloat16, false>(a, s);
  return a.dh ? norm::launch_backward<float, true>(a, s) : norm::launch_backward<float, false>(a, s);
}

}  // namespace qmm
