// What the kernels of attention over the 8-bit key-value cache share: how the work is
// cut and how its parts are joined.
#pragma once

#include <atomic>

#include "chain.cuh"
#include "common.cuh"
#include "kv.cuh"

namespace qmm {

constexpr float kKvMax = 3.402823466e38f;   // the largest float32
constexpr float kKvNone = -kKvMax;     // a running maximum that has seen nothing: no score may lie below it
constexpr float kKvSlack = 8.f;        // how far a score may pass the running maximum (a factor of 256)

// A part of an item that one warp (in shared memory) or one CTA (in the workspace) holds.
enum { kPartNone = 0, kPartHeld = 1, kPartBegins = 2, kPartEnds = 4 };
struct alignas(16) KvPart {
  int start, h;       // the sequence's first packed row, the key head
  int first, rows;    // the tile's first row (of those of one key head) and how many it has
  int flags, pad[3];
};

__host__ __device__ constexpr size_t kv_part_bytes(int dim, int rows) { return (size_t)rows * (dim + 2) * 4; }

struct KvWork {
  KvAttentionArgs a;
  long long rows_from, rows_to;   // this kernel takes the sequences with so many rows a key head
  KvPart* parts;                  // [ctas][2]
  uint8_t* ws;                    // [ctas][2] parts of kRows * (D + 2) floats
  int ctas;
};

// The kernel for many rows (kv_attention_tiles.cu): of all sequences, or, where `few` is
// the work that the rows kernel has done of the same call, of those with more rows than
// it takes (whose parts are then joined with this kernel's).
size_t kv_tiles_workspace(int head_dim, bool bf16);
cudaError_t launch_kv_attention_tiles(const KvAttentionArgs& a, const KvWork* few, void* workspace, int head_dim, bool bf16,
                                      bool vec, cudaStream_t s);

// The kernels cut the work of a call alike: all (sequence, tile of R rows, key head)
// items end to end in units of TK tokens, and to each worker the same number of
// consecutive units, wherever items begin and end. The first E units of an item stand
// for what an item costs beside its tokens, and hold none.

// The units of one row tile: at least one of tokens, so that rows that see nothing are
// written.
template <int R, int TK, int E>
__device__ __forceinline__ int kv_tile_units(const KvWork& w, const KvSeq& s, int r) {
  const int last = min((int)(((unsigned)(r + 1) * R - 1) / (unsigned)w.a.group), s.n - 1);
  return max((kv_visible(s, last, w.a.causal) + (TK - 1u)) / TK, 1u) + E;
}
template <int R>
__device__ __forceinline__ int kv_tile_count(const KvWork& w, const KvSeq& s) {
  const long long rows = (long long)s.n * w.a.group;
  return rows < w.rows_from || rows > w.rows_to ? 0 : (int)((rows + R - 1) / R);
}

// The units of sequence b, another one in each lane; a whole warp calls. A sequence of
// many row tiles is summed by all lanes.
template <int R, int TK, int E>
__device__ __forceinline__ long long kv_sequence_units(const KvWork& w, int b) {
  const int lane = threadIdx.x & 31;
  KvSeq s{};
  int tiles = 0;
  if (b < w.a.batch.batch) {
    s = kv_sequence(w.a.batch, b);
    tiles = kv_tile_count<R>(w, s);
  }
  long long sum = 0;
  if (tiles <= 2)
    for (int r = 0; r < tiles; ++r) sum += kv_tile_units<R, TK, E>(w, s, r);
  for (unsigned many = __ballot_sync(~0u, tiles > 2); many; many &= many - 1) {
    const int l = __ffs(many) - 1;
    KvSeq o{};
    o.n = __shfl_sync(~0u, s.n, l);
    o.len = __shfl_sync(~0u, s.len, l);
    o.seen = __shfl_sync(~0u, s.seen, l);
    const int count = __shfl_sync(~0u, tiles, l);
    long long all = 0;
    for (int r = lane; r < count; r += 32) all += kv_tile_units<R, TK, E>(w, o, r);
#pragma unroll
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(~0u, all, d);
    if (lane == l) sum = all;
  }
  return sum * w.a.cache.heads;
}
// Inclusive prefix sums over the lanes.
__device__ __forceinline__ long long kv_prefix(long long mine) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(~0u, mine, o);
    if (lane >= o) mine += up;
  }
  return mine;
}
// The first lane whose prefix sum passes `place`, or -1; `place` counts from that lane's
// own beginning, or from the end of them all.
__device__ __forceinline__ int kv_find(long long mine, long long incl, long long& place) {
  const unsigned past = __ballot_sync(~0u, incl > place);
  const int l = past ? __ffs(past) - 1 : 31;
  place -= __shfl_sync(~0u, past ? incl - mine : incl, l);
  return past ? l : -1;
}

// A place in the line of units.
template <int R, int TK, int E>
struct KvCursor {
  int b, r, h, at, units, tiles;   // unit `at` of `units` of the item (b, r, h)
  KvSeq s;

  // The line cut for `workers`, shares of no less than `least` units: to the beginning of
  // the index-th share, whose length is returned (0: there is none). A whole warp calls.
  __device__ long long open(const KvWork& w, int workers, int least, int index) {
    const int lane = threadIdx.x & 31, batch = w.a.batch.batch;
    const long long mine = kv_sequence_units<R, TK, E>(w, lane), incl = kv_prefix(mine);
    long long total = 0;
    for (int b0 = 32; b0 < batch; b0 += 32) total += kv_sequence_units<R, TK, E>(w, b0 + lane);
    if (batch > 32) {
#pragma unroll
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    }
    total += __shfl_sync(~0u, incl, 31);
    const long long more = total + workers - 1;
    const long long share = max(more >> 32 ? more / workers : (long long)((unsigned)more / (unsigned)workers),
                                (long long)least);
    long long place = share * index;
    const long long count = min(total - place, share);
    if (count <= 0) return 0;
    b = kv_find(mine, incl, place);
    for (int b0 = 32; b < 0 && b0 < batch; b0 += 32) {
      const long long u = kv_sequence_units<R, TK, E>(w, b0 + lane);
      const int l = kv_find(u, kv_prefix(u), place);
      if (l >= 0) b = b0 + l;
    }
    s = kv_sequence(w.a.batch, b);
    tiles = kv_tile_count<R>(w, s);
    r = 0;
    for (int r0 = 0; tiles > 1 && r0 < tiles; r0 += 32) {
      const long long u =
          r0 + lane < tiles ? (long long)kv_tile_units<R, TK, E>(w, s, r0 + lane) * w.a.cache.heads : 0;
      const int l = kv_find(u, kv_prefix(u), place);
      if (l >= 0) {
        r = r0 + l;
        break;
      }
    }
    units = kv_tile_units<R, TK, E>(w, s, r);
    h = place >> 32 ? (int)(place / units) : (int)((unsigned)place / (unsigned)units);
    at = (int)(place - (long long)h * units);
    return count;
  }
  // To the next item's first unit.
  __device__ void next_item(const KvWork& w) {
    at = 0;
    if (++h < w.a.cache.heads) return;
    h = 0;
    if (++r >= tiles) {
      r = 0;
      do {
        if (++b >= w.a.batch.batch) return;
        s = kv_sequence(w.a.batch, b);
        tiles = kv_tile_count<R>(w, s);
      } while (tiles == 0);
    }
    units = kv_tile_units<R, TK, E>(w, s, r);
  }
};

// Where a row goes: a sequence's rows of a key head are (token, query head of the
// group), token major.
__device__ __forceinline__ long long kv_out_row(const KvAttentionArgs& a, int start, int h, int row) {
  const int token = (unsigned)row / (unsigned)a.group;
  return (long long)(start + token) * ((long long)a.cache.heads * a.group) + (long long)h * a.group +
         (row - token * a.group);
}

// Parts [first, first + count) of one item joined, one row by one warp: halves of rows of
// O that are already divided by their own sums l, with their maxima m. part(i) gives the
// i-th part's bytes. The joined row is written to `out` (T, row index given) where it
// is the whole item's, else as a part again.
// Every sum is a mean, weights that add up to 1, and the parts are halved, because values
// reach up to the end of float32's range: one that is stored as 64 * 2^122 lies just past
// it, and is a row's own only where it is all that the row sees.
constexpr float kKvPartScale = 0.5f;
template <int D, typename T, typename F>
__device__ __forceinline__ void kv_join_row(int count, int rows, int row, F part, bool whole, T* out, uint8_t* into) {
  constexpr int kE = D / 32;
  const int lane = threadIdx.x & 31;
  float top = kKvNone, sum = 0.f, acc[kE] = {};
  constexpr int kAhead = 4;   // parts loaded together
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += kAhead) {
    float2 ml[kAhead];
    float x[kAhead][kE];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      ml[j] = make_float2(kKvNone, 0.f);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[j][e] = 0.f;
      const uint8_t* p = part(min(i0 + j, count - 1));
      if (i0 + j < count) {
        ml[j] = reinterpret_cast<const float2*>(p + rows * D * 4)[row];
        if constexpr (kE == 4) {
          const float4 v = reinterpret_cast<const float4*>(p)[row * 32 + lane];
          x[j][0] = v.x; x[j][1] = v.y; x[j][2] = v.z; x[j][3] = v.w;
        } else {
          const float2 v = reinterpret_cast<const float2*>(p)[row * 32 + lane];
          x[j][0] = v.x; x[j][1] = v.y;
        }
      }
    }
    float up = top;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) up = fmaxf(up, ml[j].x);
    const float down = exp2f(top - up);
    top = up;
    const float before = sum * down;
    sum = before;
    float weight[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      weight[j] = ml[j].y * exp2f(ml[j].x - top);
      sum += weight[j];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum, keep = before * inv;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= keep;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] += weight[j] * inv * x[j][e];
    }
  }
  if (whole) {
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= 1.f / kKvPartScale;
  }
  if (!whole) {
    float* o = reinterpret_cast<float*>(into) + row * D + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = acc[e];
    if (lane == 0) reinterpret_cast<float2*>(into + rows * D * 4)[row] = make_float2(top, sum);
  } else if (out) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < kE; ++e) out[lane * kE + e] = acc[e];
    } else {
      uint32_t u[kE / 2];
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
      if constexpr (kE == 4) {
        *reinterpret_cast<uint2*>(out + lane * 4) = make_uint2(u[0], u[1]);
      } else {
        *reinterpret_cast<uint32_t*>(out + lane * 2) = u[0];
      }
    }
  }
}

// What several CTAs hold of an item, joined by the CTAs with the number of the one that
// holds its beginning: slice `slice` of `slices` of its rows.
template <int D, int R, typename T>
__device__ __forceinline__ void kv_join_parts(const KvWork& w, int slice, int slices) {
  if ((int)blockIdx.x >= w.ctas) return;
  const KvPart a = w.parts[2 * blockIdx.x + 1];
  if (!(a.flags & kPartHeld)) return;
  // the following CTAs' first parts belong to the item, up to the one that ends it
  const int lane = threadIdx.x & 31;
  int n = 1;
  for (int c0 = blockIdx.x + 1; c0 < w.ctas; c0 += 32) {
    const int c = c0 + lane;
    const unsigned ends = __ballot_sync(~0u, c < w.ctas && (w.parts[2 * c].flags & kPartEnds));
    if (ends) {
      n += __ffs(ends);
      break;
    }
    n += 32;
  }
  n = min(n, w.ctas - (int)blockIdx.x);
  auto part = [&](int j) -> const uint8_t* {
    return w.ws + (size_t)(j == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + j)) * kv_part_bytes(D, R);
  };
  for (int row = slice * 8 + (threadIdx.x >> 5); row < a.rows; row += 8 * slices) {
    T* out = static_cast<T*>(w.a.out) + kv_out_row(w.a, a.start, a.h, a.first + row) * D;
    kv_join_row<D, T>(n, R, row, part, true, out, nullptr);
  }
}
template <int D, int R, typename T>
__global__ void __launch_bounds__(256) kv_attention_join_kernel(const KvWork w) {
  chain_wait();
  kv_join_parts<D, R, T>(w, blockIdx.y, gridDim.y);
  chain_release();
}
// The parts of both kernels in one launch: `few` by the last slice of the grid.
template <int D, int RFew, int RMany, typename T>
__global__ void __launch_bounds__(256) kv_attention_join_both_kernel(const KvWork few, const KvWork many) {
  chain_wait();
  if (blockIdx.y + 1 == gridDim.y) {
    kv_join_parts<D, RFew, T>(few, 0, 1);
  } else {
    kv_join_parts<D, RMany, T>(many, blockIdx.y, gridDim.y - 1);
  }
  chain_release();
}

// The opt-in to a kernel's shared memory, once a device.
template <auto kern>
cudaError_t kv_allow_smem(int bytes) {
  static std::atomic<bool> done[64];
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (done[device].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[device].store(true, std::memory_order_relaxed);
  return e;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What is left of a and b beside their fp16 pair, in fp16.
__device__ __forceinline__ uint32_t half_rest(float a, float b, uint32_t pair) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&pair));
  return half_pair(a - h.x, b - h.y);
}
// The values' powers of two. P, in fp16, has few digits to spare for them: times 2^30 for
// a block that a row hardly sees, or does not see, the P of all that it does see would
// be zeros. So they go into the fp16 that an int8 of V becomes, at no cost (kv_widen):
// int8 * 2^(byte - window), exactly, for bytes from `below` under the window's to kKvAbove
// over it. A window holds for as long as the bytes stay within. Where they do not, it
// moves, and a row that takes part in a block of another window has its O rescaled from
// unit to unit. Rows that see nothing of the block are left alone: what they add, 0 * V, is
// 0 in any unit.
// P is held by the row's largest score, not by its largest score * value, which may be as
// much smaller as a window is wide: of the 31 binades that it has below 2^7, bfloat16's
// leaves 13 to the digits of what weighs most, float32's 21.
constexpr int kKvAbove = 5, kKvNoWindow = -1000;
template <typename T>
constexpr int kKvBelow = sizeof(T) == 4 ? 5 : 13;
__host__ __device__ constexpr bool kv_in_window(int byte, int window, int below) {
  return byte >= window - below && byte <= window + kKvAbove;
}
// The window around bytes lo .. hi, which are no further apart than it holds. (Between 1 and 250, 2^(window - 127) is
// a normal number, and bytes 0 and 255 are still within.)
__host__ __device__ constexpr int kv_window(int lo, int hi, int below) {
  const int w = (lo + hi + below - kKvAbove + 1) / 2;
  return w < 1 ? 1 : w > 250 ? 250 : w;
}
// The window that holds lo .. hi and is next to the one that there is, so that windows of a sequence settle.
__host__ __device__ constexpr int kv_move_window(int window, int lo, int hi, int below) {
  return window == kKvNoWindow      ? kv_window(lo, hi, below)
         : window < hi - kKvAbove   ? hi - kKvAbove
         : window > lo + below      ? lo + below
                                    : window;
}
template <int below>
constexpr bool kKvWindowHolds = kv_in_window(0, kv_window(0, 0, below), below) &&
                                kv_in_window(255, kv_window(255, 255, below), below) &&
                                kv_in_window(0, kv_window(0, below + 5, below), below) &&
                                kv_in_window(below + 5, kv_window(0, below + 5, below), below) &&
                                kv_in_window(101, kv_window(101, 106 + below, below), below) &&
                                kv_in_window(106 + below, kv_window(101, 106 + below, below), below) &&
                                kv_in_window(250 - below, kv_window(250 - below, 255, below), below) &&
                                kv_in_window(255, kv_window(250 - below, 255, below), below);
static_assert(kKvWindowHolds<5> && kKvWindowHolds<13>, "a window holds what it was made for");

// A row's units: P is held in 2^m, O in 2^(m + window), the sum l in 2^(m - behind), that
// is by the largest score so far. behind is 0 but where windows moved: below 0 for a block
// with low scores, whose P has to be held by its own, above 0 for a block so far below
// the last ones that O could not follow.
struct KvUnit {
  float m, behind;
  int window;
};
// P and l of a row far above its scores: P is 0 in fp16 2^40 above them; no further than this, so that float32 still
// holds what l takes from it.
constexpr float kKvFar = 100.f;
// A factor to O, of which one float32 holds half the range.
struct KvFactor {
  float a, b;   // b: 1 but for factors below 2^-126
};
// The row comes to scores of which the largest is top (-inf: it sees none of them), with
// values in `window`. `largest`: of its O, in magnitude. Returns the factor to O; l is
// taken to its unit here.
__device__ __forceinline__ KvFactor kv_change_units(KvUnit& u, float& l, float top, float largest, int window) {
  const float most = u.m - u.behind, unit = fmaxf(most, top);   // of l: before, after
  if (top > most) l *= exp2_approx(most - top);
  float up = fmaxf(u.m, top), shift = u.m - up;
  if (top > -INFINITY && u.window != window) {
    up = top > unit - 2.f ? unit : top;
    shift = 0.f;
    if (largest > 0.f) {
      const float moves = (float)(u.window - window);
      const float room = fminf(251.f - (float)(__float_as_int(largest) >> 23), 126.f);   // O stays below 2^125
      up = fmaxf(up, u.m + moves - room);
      shift = u.m - up + moves;
    }
    u.window = window;
    u.behind = up - unit;
  } else if (top > most || up > u.m) {
    u.behind = up - unit;
  }
  u.m = up;
  const float held = fmaxf(shift, -126.f);
  return {exp2_approx(held), exp2_approx(shift - held)};
}

// Two int8, biased by 128, to two fp16: bytes 0 and 1 of u, or 2 and 3. The byte becomes
// the low mantissa bits of 1024, whose ulp is 1, and 1024 + 128 is taken off, exactly.
__device__ __forceinline__ uint32_t bytes_low(uint32_t u) {
  const uint32_t l = prmt(u, 0x64646464u, 0x4140u);
  const __half2 bias(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bytes_high(uint32_t u) {
  const uint32_t l = prmt(u, 0x64646464u, 0x4342u);
  const __half2 bias(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The same times 2^s, s from -14 to kKvAbove, exactly: (1152 + int8) * 2^s - 1152 * 2^s in one operation.
struct alignas(8) KvScale {
  uint32_t factor, bias;   // fp16 pairs: 2^s, -1152 * 2^s
};
__device__ __forceinline__ KvScale kv_scale(int s) {
  return {((uint32_t)(s + 15) << 10) * 0x10001u, (0x8080u + ((uint32_t)(s + 25) << 10)) * 0x10001u};
}
__device__ __forceinline__ uint32_t kv_widen(uint32_t biased, KvScale k) {
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&biased), *reinterpret_cast<const __half2*>(&k.factor),
                            *reinterpret_cast<const __half2*>(&k.bias));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bytes_low(uint32_t u, KvScale k) { return kv_widen(prmt(u, 0x64646464u, 0x4140u), k); }
__device__ __forceinline__ uint32_t bytes_high(uint32_t u, KvScale k) { return kv_widen(prmt(u, 0x64646464u, 0x4342u), k); }

}  // namespace qmm
