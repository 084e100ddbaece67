// The 8-bit key-value cache: appending keys and values (keys and queries rotated to
// their positions on the way), and reading tokens back. Format: include/qmm.h.
//
// Both are passes over memory: what is read and written once is all the work, so the
// layout of threads follows the rows. A warp of the append owns one block of 16
// tokens of one head, of keys or of values, in registers: the block's largest
// magnitude, which decides its power of two, is then a warp's reduction, and nobody
// else writes that block. A lane holds two groups of eight elements that a rotation
// pairs (element i with i + half, or neighbours), so that the pair meets in one lane.
//
// Measured: 8192 tokens of 64 query and 8 + 8 key and value heads of 128, bfloat16, 60 us
// (319 MB: 79 % of a copy's rate) and 14 us for reading them back (50 MB, 53 %); one token
// of each of 256 sequences about 8 and 7 us, most of it loads that follow each other.
#include "chain.cuh"
#include "kv.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPasses = 4;               // of heads, by a warp that rotates queries

// Where a lane's two groups of eight begin in a head: li = 0 .. dim / 16 - 1.
struct Groups {
  int a, b;     // first elements
  int turn;     // first row entry of cos and sin that rotates them, or -1
};
__device__ __forceinline__ Groups groups_of(int li, int half, int interleaved) {
  if (interleaved) return {16 * li, 16 * li + 8, 16 * li < 2 * half ? 8 * li : -1};
  if (8 * li < half) return {8 * li, 8 * li + half, 8 * li};
  const int d = 2 * half + 16 * (li - half / 8);
  return {d, d + 8, -1};
}

// (a, b) -> (a c - b s, b c + a s), every product rounded to float32 by itself.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}
__device__ __forceinline__ void turn_groups(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8],
                                            int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
      turn_pair(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], c[i], s[i]);
  }
}
// Eight entries of cos and sin of position pos; NaN for a position without a row.
__device__ __forceinline__ void load_turn(const KvAppendArgs& p, int pos, int at, float (&c)[8], float (&s)[8]) {
  if (pos < 0 || pos >= p.positions) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
    return;
  }
  const size_t o = (size_t)pos * p.half + at;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p.cos + o + i));
    const float4 y = __ldg(reinterpret_cast<const float4*>(p.sin + o + i));
    c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
    s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
  }
}

// What the cache stores of a number that is not finite: nothing of a NaN, the largest
// finite number for an infinity.
__device__ __forceinline__ float storable(float x) {
  constexpr float kMax = 3.402823466e38f;
  return x == x ? fminf(fmaxf(x, -kMax), kMax) : 0.f;
}

// Four int8, clamped to +-127, in one word.
__device__ __forceinline__ uint32_t pack4(const float* x, float up) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = min(max(__float2int_rn(x[i] * up), -127), 127);
    w |= (uint32_t)(q & 255) << (8 * i);
  }
  return w;
}
// Four int8 times 2^-shift, to nearest even.
__device__ __forceinline__ uint32_t shift4(uint32_t w, float down) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = __float2int_rn((float)(int8_t)(w >> (8 * i)) * down);
    r |= (uint32_t)(q & 255) << (8 * i);
  }
  return r;
}

// One block of 16 tokens of one head, by one warp. base: its first token; new tokens
// are [from, to) of the sequence, the ones before `from` are kept.
template <int D, typename T, bool kVec>
__device__ __forceinline__ void append_block(const KvAppendArgs& p, const KvSeq& s, int base, int from, int to,
                                             size_t block, const T* x, long long row_stride, int8_t* cache,
                                             uint8_t* exps, bool rotate) {
  constexpr int kLanes = D / 16;          // lanes of a token
  constexpr int kTokens = 32 / kLanes;    // tokens a pass
  constexpr int kSteps = kKvBlock / kTokens;
  const int lane = threadIdx.x & 31;
  const int li = lane % kLanes, ti = lane / kLanes;
  const Groups g = groups_of(li, rotate ? p.half : 0, rotate && p.interleaved);
  // The block stays as it was read: it is rotated once for its largest magnitude and once more to be stored, which
  // costs less than the registers of 64 numbers a lane would (a third fewer warps on an SM).
  KvRaw<T> ra[kSteps], rb[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int pos = base + i * kTokens + ti;
    if (pos >= from && pos < to) {
      const T* r = x + (long long)(s.start + (pos - (s.len - s.n))) * row_stride;
      ra[i].template load<kVec>(r + g.a);
      rb[i].template load<kVec>(r + g.b);
    }
  }
  auto step = [&](int i, float (&a)[8], float (&b)[8]) {
    ra[i].floats(a);
    rb[i].floats(b);
    if (rotate && g.turn >= 0) {
      float c[8], sn[8];
      load_turn(p, base + i * kTokens + ti, g.turn, c, sn);
      turn_groups(a, b, c, sn, p.interleaved);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = storable(a[e]);
      b[e] = storable(b[e]);
    }
  };
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int pos = base + i * kTokens + ti;
    if (pos >= from && pos < to) {
      float a[8], b[8];
      step(i, a, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(a[e]), fabsf(b[e])));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  int byte = kv_exponent(top);
  const bool live = base < from;
  int held = 0;
  if (live) {
    held = exps[block];
    byte = max(byte, held);
  }
  const float up = kv_power(254 - byte);
  const float down = kv_power(127 - min(byte - held, 20));
  int8_t* c = cache + block * (size_t)(kKvBlock * D);
  __syncwarp();   // every lane has read the byte
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int pos = base + i * kTokens + ti;
    int8_t* r = c + (i * kTokens + ti) * D;
    if (pos >= from && pos < to) {
      float a[8], b[8];
      step(i, a, b);
      *reinterpret_cast<uint2*>(r + g.a) = make_uint2(pack4(a, up), pack4(a + 4, up));
      *reinterpret_cast<uint2*>(r + g.b) = make_uint2(pack4(b, up), pack4(b + 4, up));
    } else if (pos < from && byte > held) {
      // the block's scale grows: the tokens that are there follow it
      uint2 u = *reinterpret_cast<const uint2*>(r + g.a), w = *reinterpret_cast<const uint2*>(r + g.b);
      *reinterpret_cast<uint2*>(r + g.a) = make_uint2(shift4(u.x, down), shift4(u.y, down));
      *reinterpret_cast<uint2*>(r + g.b) = make_uint2(shift4(w.x, down), shift4(w.y, down));
    }
  }
  if (lane == 0) exps[block] = (uint8_t)byte;
}

// CTAs [0, slots * slot_ctas): the cache. Slot w holds one block of one sequence:
// sequence b owns the slots from floor(starts[b] / 16) + 2 b on, which leaves room for
// the floor(n / 16) + 2 blocks that n tokens can touch, so that the slot count follows
// from the rows and the batch alone. The slot's warps are its heads, keys first. The
// CTAs behind those rotate queries: a warp takes one token and up to four passes of heads,
// whose loads go out before it looks for the token's position.
template <int D, typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) kv_append_kernel(const KvAppendArgs p) {
  chain_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.cache.heads;
  const long long cache_ctas = (long long)p.slots * p.slot_ctas;
  if ((long long)blockIdx.x < cache_ctas) {
    const int w = blockIdx.x / p.slot_ctas;
    const int task = (blockIdx.x % p.slot_ctas) * kWarps + warp;
    if (task < 2 * heads) {
      int b = w, first = 0;
      if (p.batch.starts) {
        // the last sequence whose slots begin at w or before
        int count = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.batch.batch; b0 += 128) {
          int begins[4];   // four loads in flight
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = b0 + 32 * e + lane;
            begins[e] = i < p.batch.batch ? (max(__ldg(p.batch.starts + i), 0) >> 4) + 2 * i : INT_MAX;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) count += __popc(__ballot_sync(~0u, begins[e] <= w));
        }
        b = count - 1;
        if (b >= 0) first = w - ((max(__ldg(p.batch.starts + b), 0) >> 4) + 2 * b);
      }
      if (b >= 0) {
        const KvSeq s = kv_sequence(p.batch, b);
        const int p0 = max(s.len - s.n, 0);
        const long long from_base = (long long)(p0 / kKvBlock + first) * kKvBlock;
        if (s.n > 0 && first >= 0 && from_base < s.seen) {
          const int base = (int)from_base, blk = base / kKvBlock;
          const int page = __ldg(p.batch.table + (size_t)b * p.batch.width + blk / p.cache.bpp);
          if (page >= 0 && page < p.cache.pages) {
            const bool key = task < heads;
            const int h = key ? task : task - heads;
            const size_t block = ((size_t)page * heads + h) * p.cache.bpp + blk % p.cache.bpp;
            const int from = max(p0, base), to = base + min(s.seen - base, kKvBlock);
            if (key) {
              append_block<D, T, kVec>(p, s, base, from, to, block,
                                       static_cast<const T*>(p.k) + (long long)h * p.k_head, p.k_row, p.cache.k,
                                       p.cache.ke, p.half > 0);
            } else {
              append_block<D, T, kVec>(p, s, base, from, to, block,
                                       static_cast<const T*>(p.v) + (long long)h * p.v_head, p.v_row, p.cache.v,
                                       p.cache.ve, false);
            }
          }
        }
      }
    }
    chain_release();
    return;
  }
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;   // heads a pass
  const int chunks = (p.q_heads + kPasses * kHeads - 1) / (kPasses * kHeads);
  const long long task = ((long long)blockIdx.x - cache_ctas) * kWarps + warp;
  if (task < (long long)p.batch.rows * chunks) {
    const int t = (int)((unsigned long long)task / (unsigned)chunks), chunk = (int)(task - (long long)t * chunks);
    const int li = lane % kLanes;
    const Groups g = groups_of(li, p.half, p.interleaved);
    const int h0 = chunk * kPasses * kHeads + lane / kLanes;
    // the rows first, which need no position
    KvRaw<T> ra[kPasses], rb[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int h = h0 + i * kHeads;
      if (h < p.q_heads) {
        const T* r = static_cast<const T*>(p.q) + (long long)t * p.q_row + (long long)h * p.q_head;
        ra[i].template load<kVec>(r + g.a);
        rb[i].template load<kVec>(r + g.b);
      }
    }
    const int b = kv_sequence_of_row(p.batch, t);
    if (b >= 0) {
      const KvSeq s = kv_sequence(p.batch, b);
      if (t >= s.start && t < s.start + s.n) {
        float c[8], sn[8];
        if (g.turn >= 0) load_turn(p, s.len - s.n + (t - s.start), g.turn, c, sn);
        chain_release();
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int h = h0 + i * kHeads;
          if (h < p.q_heads) {
            float a[8], e[8];
            ra[i].floats(a);
            rb[i].floats(e);
            if (g.turn >= 0) turn_groups(a, e, c, sn, p.interleaved);
            T* r = static_cast<T*>(p.q_out) + ((size_t)t * p.q_heads + h) * D;
            kv_store8(r + g.a, a);
            kv_store8(r + g.b, e);
          }
        }
        return;
      }
    }
  }
  chain_release();
}

// A warp reads one token back: a lane takes 16 int8 of a head.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs p) {
  chain_wait();
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t < p.batch.rows) {
    const int b = kv_sequence_of_row(p.batch, t);
    if (b >= 0) {
      const KvSeq s = kv_sequence(p.batch, b);
      if (t >= s.start && t < s.start + s.n) {
        const int pos = s.len - s.n + (t - s.start);
        int page = -1, blk = 0;
        if (pos >= 0 && pos < s.seen) {
          blk = pos / kKvBlock;
          page = __ldg(p.batch.table + (size_t)b * p.batch.width + blk / p.cache.bpp);
          if (page >= p.cache.pages) page = -1;
        }
        const int li = lane % kLanes;
        for (int h = lane / kLanes; h < p.cache.heads; h += kHeads) {
          const size_t block = page < 0 ? 0 : ((size_t)page * p.cache.heads + h) * p.cache.bpp + blk % p.cache.bpp;
          const size_t at = block * (kKvBlock * D) + (pos % kKvBlock) * D + 16 * li;
          const size_t to = ((size_t)t * p.cache.heads + h) * D + 16 * li;
#pragma unroll
          for (int kind = 0; kind < 2; ++kind) {
            T* out = static_cast<T*>(kind ? p.v : p.k);
            if (!out) continue;
            uint4 w = make_uint4(0, 0, 0, 0);
            float step = 0.f;
            if (page >= 0) {
              w = *reinterpret_cast<const uint4*>((kind ? p.cache.v : p.cache.k) + at);
              step = kv_power((kind ? p.cache.ve : p.cache.ke)[block]);
            }
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            float x[2][8];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e / 8][e % 8] = (float)(int8_t)(u[e / 4] >> (8 * (e % 4))) * step;
            kv_store8(out + to, x[0]);
            kv_store8(out + to + 8, x[1]);
          }
        }
      }
    }
  }
  chain_release();
}

template <int D, typename T>
cudaError_t append_typed(KvAppendArgs a, bool vec, cudaStream_t s) {
  a.slots = a.batch.starts ? a.batch.rows / kKvBlock + 2 * a.batch.batch : a.batch.batch;
  a.slot_ctas = (2 * a.cache.heads + kWarps - 1) / kWarps;
  constexpr int kHeads = 32 / (D / 16);
  const long long chunks = (a.q_heads + kPasses * kHeads - 1) / (kPasses * kHeads);
  const long long q_ctas = a.q ? (a.batch.rows * chunks + kWarps - 1) / kWarps : 0;
  const long long grid = (long long)a.slots * a.slot_ctas + q_ctas;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  auto kern = vec ? &kv_append_kernel<D, T, true> : &kv_append_kernel<D, T, false>;
  return launch_chained(kern, dim3((unsigned)grid), dim3(kThreads), 0, 1, s, a);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int head_dim, bool bf16, bool vec, cudaStream_t s,
                             const char** kernel_name) {
  *kernel_name = "kv_append";
  if (head_dim == 64)
    return bf16 ? append_typed<64, __nv_bfloat16>(a, vec, s) : append_typed<64, float>(a, vec, s);
  return bf16 ? append_typed<128, __nv_bfloat16>(a, vec, s) : append_typed<128, float>(a, vec, s);
}

cudaError_t launch_kv_read(const KvReadArgs& a, int head_dim, bool bf16, cudaStream_t s, const char** kernel_name) {
  *kernel_name = "kv_read";
  const dim3 grid((a.batch.rows + kWarps - 1) / kWarps), block(kThreads);
  if (head_dim == 64)
    return bf16 ? launch_chained(&kv_read_kernel<64, __nv_bfloat16>, grid, block, 0, 1, s, a)
                : launch_chained(&kv_read_kernel<64, float>, grid, block, 0, 1, s, a);
  return bf16 ? launch_chained(&kv_read_kernel<128, __nv_bfloat16>, grid, block, 0, 1, s, a)
              : launch_chained(&kv_read_kernel<128, float>, grid, block, 0, 1, s, a);
}

}  // namespace qmm
