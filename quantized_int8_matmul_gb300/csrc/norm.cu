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
// Sums and statistics are fp32. Both are bound by HBM: every tensor is read or
// written once, the row held in registers between its reduction and its output.
#include "common.cuh"
#include "kernels.h"

#include <algorithm>

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

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// E consecutive elements of a row starting at element i (VEC: one 16-byte
// access; otherwise element by element, those at or past n read as 0).
template <typename T, bool VEC>
__device__ __forceinline__ void load_e(const T* row, int i, int n, float* v) {
  constexpr int E = Vec<T>::E;
  if (VEC) {
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(row + i), v);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = i + e < n ? to_f(row[i + e]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_e(T* row, int i, int n, const float* v) {
  constexpr int E = Vec<T>::E;
  if (VEC) {
    *reinterpret_cast<uint4*>(row + i) = Vec<T>::pack(v);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (i + e < n) row[i + e] = from_f<T>(v[e]);
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_w(const void* w, int w_f32, int i, int n, float* v) {
  constexpr int E = Vec<T>::E;
  if (w_f32) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (VEC || i + e < n) ? __ldg(static_cast<const float*>(w) + i + e) : 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = (VEC || i + e < n) ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i + e]) : 0.f;
  }
}

// Sum of a and maximum of b over the CTA (every thread gets both).
__device__ __forceinline__ void block_sum_max(float& a, unsigned& b) {
  __shared__ float sa[32];
  __shared__ unsigned sb[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  b = __reduce_max_sync(0xffffffffu, b);
  if (nw == 1) return;
  __syncthreads();   // an earlier use of the arrays is over
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

// The row's scale and the multiplier of v. A row that holds a NaN or an
// infinity gets a NaN scale (and zeros); a row with a below 2^-100 (whose
// 127 / a could overflow, and whose squares underflow) is stored as zeros, scale 1.
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
__device__ __forceinline__ int quant1(float v, float inv) {
  const float p = fminf(fmaxf(__fmul_rn(v, inv), -127.f), 127.f);
  return __float2int_rn(p);
}

template <typename T, bool VEC>
__global__ void rms_norm_s8_kernel(const NormArgs p) {
  constexpr int E = Vec<T>::E;
  const int n = p.H, nt = blockDim.x;
  for (long long m = blockIdx.x; m < p.M; m += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + m * p.ldx;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + m * p.ldr : nullptr;
    T* ho = p.h ? static_cast<T*>(p.h) + m * (long long)n : nullptr;
    int8_t* q = p.q + m * (long long)n;
    float ss = 0.f;
    unsigned am = 0u;
    for (int i = threadIdx.x * E; i < n; i += nt * E) {
      float h[E], w[E];
      load_e<T, VEC>(x, i, n, h);
      if (r) {
        float b[E];
        load_e<T, VEC>(r, i, n, b);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = to_f(from_f<T>(__fadd_rn(h[e], b[e])));
      }
      if (ho) store_e<T, VEC>(ho, i, n, h);
      load_w<T, VEC>(p.w, p.w_f32, i, n, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ss = __fmaf_rn(h[e], h[e], ss);
        am = max(am, __float_as_uint(__fmul_rn(h[e], w[e])) & 0x7fffffffu);
      }
    }
    block_sum_max(ss, am);
    const RowScale s = row_scale(ss, am, n, p.eps);
    if (threadIdx.x == 0) {
      p.scale[m] = s.scale;
      p.rstd[m] = s.rstd;
    }
    for (int i = threadIdx.x * E; i < n; i += nt * E) {
      float h[E], w[E];
      // a stored h is read back (it may lie over x or the residual)
      load_e<T, VEC>(ho ? ho : x, i, n, h);
      if (r && !ho) {
        float b[E];
        load_e<T, VEC>(r, i, n, b);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = to_f(from_f<T>(__fadd_rn(h[e], b[e])));
      }
      load_w<T, VEC>(p.w, p.w_f32, i, n, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (VEC || i + e < n) q[i + e] = am >= kInfBits ? 0 : (int8_t)quant1(__fmul_rn(h[e], w[e]), s.inv);
      }
    }
  }
}

template <typename T>
__global__ void s8_dequantize_rows_kernel(const int8_t* q, const float* scale, long long M, int H, T* y) {
  const long long m = blockIdx.x;
  const float s = scale[m];
  for (int i = threadIdx.x; i < H; i += blockDim.x)
    y[m * H + i] = from_f<T>(__fmul_rn((float)q[m * H + i], s));
}

template <typename T>
__global__ void rms_norm_backward_kernel(const NormBwdArgs p) {
  const int n = p.H, nt = blockDim.x;
  float* part = p.partials + (long long)blockIdx.x * n;
  for (int i = threadIdx.x; i < n; i += nt) part[i] = 0.f;
  for (long long m = blockIdx.x; m < p.M; m += gridDim.x) {
    const T* h = static_cast<const T*>(p.h) + m * p.ldh;
    const T* dy = static_cast<const T*>(p.dy) + m * p.lddy;
    const T* dh = p.dh ? static_cast<const T*>(p.dh) + m * p.lddh : nullptr;
    T* dx = static_cast<T*>(p.dx) + m * (long long)n;
    const float rstd = p.rstd[m];
    float dot = 0.f;
    unsigned unused = 0u;
    for (int i = threadIdx.x; i < n; i += nt) {
      float w[1];
      w[0] = p.w_f32 ? static_cast<const float*>(p.w)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[i]);
      dot = __fmaf_rn(to_f(dy[i]) * w[0], to_f(h[i]) * rstd, dot);
    }
    block_sum_max(dot, unused);
    const float mean = dot / (float)n;
    for (int i = threadIdx.x; i < n; i += nt) {
      const float w = p.w_f32 ? static_cast<const float*>(p.w)[i]
                              : __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[i]);
      const float d = to_f(dy[i]), nn = to_f(h[i]) * rstd;
      float v = rstd * (d * w - nn * mean);
      if (dh) v += to_f(dh[i]);
      dx[i] = from_f<T>(v);
      part[i] += d * nn;
    }
  }
}

__global__ void sum_partials_kernel(const float* part, int count, int n, float* out) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int c = 0; c < count; ++c) s += part[(long long)c * n + i];
  out[i] = s;
}

template <typename T>
bool rows_vec(const void* p, long long ld) {
  return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * (long long)sizeof(T)) % 16 == 0;
}

template <typename T>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  constexpr int E = Vec<T>::E;
  const bool vec = a.H % E == 0 && rows_vec<T>(a.x, a.ldx) && (!a.residual || rows_vec<T>(a.residual, a.ldr)) &&
                   (!a.h || rows_vec<T>(a.h, a.H));
  const int threads = std::min(512, std::max(32, ((a.H + E - 1) / E + 31) / 32 * 32));
  const unsigned grid = (unsigned)std::min<long long>(a.M, 1 << 30);
  if (vec) rms_norm_s8_kernel<T, true><<<grid, threads, 0, s>>>(a);
  else rms_norm_s8_kernel<T, false><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace norm

cudaError_t launch_rms_norm_s8(const NormArgs& a, bool bf16, cudaStream_t s, const char** kernel_name) {
  *kernel_name = "rms_norm_s8";
  return bf16 ? norm::launch_norm<__nv_bfloat16>(a, s) : norm::launch_norm<float>(a, s);
}

cudaError_t launch_s8_dequantize_rows(const int8_t* q, const float* scale, long long M, int H, void* y, bool bf16,
                                      cudaStream_t s, const char** kernel_name) {
  *kernel_name = "s8_dequantize_rows";
  if (bf16)
    norm::s8_dequantize_rows_kernel<<<(unsigned)M, 256, 0, s>>>(q, scale, M, H, static_cast<__nv_bfloat16*>(y));
  else
    norm::s8_dequantize_rows_kernel<<<(unsigned)M, 256, 0, s>>>(q, scale, M, H, static_cast<float*>(y));
  return cudaGetLastError();
}

int rms_norm_backward_partials(long long M, int H) { return (int)std::min<long long>(M, 2 * 152); }

cudaError_t launch_rms_norm_backward(const NormBwdArgs& a, bool bf16, cudaStream_t s, const char** kernel_name) {
  *kernel_name = "rms_norm_backward+sum_partials";
  const int parts = rms_norm_backward_partials(a.M, a.H);
  const int threads = std::min(512, std::max(32, (a.H + 31) / 32 * 32));
  if (bf16) norm::rms_norm_backward_kernel<__nv_bfloat16><<<parts, threads, 0, s>>>(a);
  else norm::rms_norm_backward_kernel<float><<<parts, threads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm::sum_partials_kernel<<<(a.H + 127) / 128, 128, 0, s>>>(a.partials, parts, a.H, a.dweight);
  return cudaGetLastError();
}

}  // namespace qmm
