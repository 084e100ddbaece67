// The 8-bit key-value cache as the kernels see it (format: include/qmm.h), and the
// packed sequences of a call.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace qmm {

constexpr int kKvBlock = 16;   // tokens that share a scale

// One sequence of a call: its packed rows and its tokens in the cache. What the
// device finds in starts and lengths is clamped to the call's rows and to the table,
// so that no index derived from them leaves either.
struct KvSeq {
  int start;   // first packed row
  int n;       // rows
  int len;     // tokens, the rows' own among them, as given (0 where negative)
  int seen;    // of those, the ones that the table has room for
};

__device__ __forceinline__ KvSeq kv_sequence(const KvBatchArgs& a, int b) {
  KvSeq s;
  int s0 = b, s1 = b + 1;
  if (a.starts) {
    s0 = __ldg(a.starts + b);
    s1 = __ldg(a.starts + b + 1);
  }
  s.start = min(max(s0, 0), a.rows);
  s.n = max(min(max(s1, 0), a.rows) - s.start, 0);   // (a difference from -2^31 would wrap)
  s.len = max(__ldg(a.lengths + b), 0);
  s.seen = min(s.len, a.capacity);
  return s;
}

// How many tokens row token i of a sequence sees.
__device__ __forceinline__ int kv_visible(const KvSeq& s, int i, int causal) {
  return causal ? min(max(s.len - s.n + i + 1, 0), s.seen) : s.seen;
}

// The sequence that packed row t belongs to, or -1; a whole warp asks for one row.
__device__ __forceinline__ int kv_sequence_of_row(const KvBatchArgs& a, int t) {
  if (!a.starts) return t < a.batch ? t : -1;
  const int lane = threadIdx.x & 31;
  int count = 0;   // starts[1 ..] that are <= t
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += 128) {
    int ends[4];   // four loads in flight
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = b0 + 32 * e + lane;
      ends[e] = b < a.batch ? __ldg(a.starts + b + 1) : INT_MAX;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) count += __popc(__ballot_sync(~0u, ends[e] <= t));
  }
  return count < a.batch ? count : -1;
}

// 2^(byte - 127); the smallest one is below float32's normal range.
__device__ __forceinline__ float kv_power(int byte) {
  return __int_as_float(byte > 0 ? byte << 23 : 0x00400000);
}
// The byte of a block with the largest magnitude amax (finite): the smallest power of
// two under which amax rounds to 127 or less (amax / step < 127.5, that is a mantissa
// below 0x7f0000 at a step six binades down).
__device__ __forceinline__ int kv_exponent(float amax) {
  return max(((__float_as_int(amax) + 0x10000) >> 23) - 6, 0);
}

// Eight consecutive elements as they lie, and as float32. kVec: on a 16-byte boundary.
template <typename T>
struct KvRaw;
template <>
struct KvRaw<__nv_bfloat16> {
  uint4 w = make_uint4(0, 0, 0, 0);
  template <bool kVec>
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (kVec) {
      w = *reinterpret_cast<const uint4*>(p);
    } else {
      const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
      w = make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16, s[4] | (uint32_t)s[5] << 16,
                     s[6] | (uint32_t)s[7] << 16);
    }
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct KvRaw<float> {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = make_float4(0.f, 0.f, 0.f, 0.f);
  template <bool kVec>
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (kVec) {
      a = reinterpret_cast<const float4*>(p)[0];
      b = reinterpret_cast<const float4*>(p)[1];
    } else {
      a = make_float4(p[0], p[1], p[2], p[3]);
      b = make_float4(p[4], p[5], p[6], p[7]);
    }
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <bool kVec, typename T>
__device__ __forceinline__ void kv_load8(const T* p, float (&x)[8]) {
  KvRaw<T> r;
  r.template load<kVec>(p);
  r.floats(x);
}
// Eight elements to a 16-byte boundary.
__device__ __forceinline__ void kv_store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void kv_store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace qmm
