// Attention over the 8-bit key-value cache for many rows: prompts, pieces of them, an
// encoder's states, on the tensor cores (tcgen05), bfloat16 queries.
//
// What bounds it is arithmetic: 4 D operations a pair of a query row and a token, on the
// tensor cores, and one exponential. A CTA takes 256 rows of one sequence and key head
// (tokens times the query heads that share the key head, so keys are converted once for
// all of them) in two tiles of 128, and walks over the tokens 128 at a time:
//
//   S = Q K^T   A = Q, B = K, both fp16 in shared memory, S fp32 in tensor memory
//   P = exp2(S c - m), fp16, written over S, as the A operand from tensor memory
//   O += P V    B = V as it lies, tokens in rows (its other major order), fp32
//
// The two tiles alternate: while the tensor cores work for one, the softmax of the
// other runs. Warps 0-3 and 4-7 hold a row a thread (its maximum and sum need no
// exchange), warps 8-11 bring int8 keys and values from their pages through registers,
// widen them to fp16, exactly, into a ring of four operands, and one thread issues the
// MMAs. A block's power of two is not multiplied into K or V: a key block's goes into
// the factor of its 16 columns of S, a value block's into the exponent of its 16 columns
// of P. The running maximum moves only past a score 8 above it (rescaling O is then
// rare); scores are masked only in tiles that some row's limit cuts.
//
// The work is cut like that of the other kernel (kv_attention.cuh), a unit being a tile
// of 128 tokens, so that short and long rows of causal prompts balance.
#include "kv_attention.cuh"

namespace qmm {
namespace {

constexpr int kRows = 256, kTokens = 128;
constexpr int kThreads = 448;
constexpr int kStages = 4;                 // operands (K or V tiles) in the ring
constexpr int kInfo = 4;                   // tiles whose scales are kept
constexpr int kBlocks = kTokens / kKvBlock;
constexpr int kMinTiles = 2;               // a CTA's share, at least
constexpr float kLift = 7.f;               // P is held times 2^7: at most 2^15

struct Info {
  float kpow[kBlocks];     // 2^(byte - 127) of the tile's key blocks
  int ve[kBlocks];         // bytes of its value blocks
  int vmax;                // the largest of them
  int missing;             // blocks on pages that are not there, a bit each
};

template <int D>
struct Smem {
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kStage = kTokens * D * 2;
  alignas(1024) uint8_t q[2 * kQTile];
  alignas(1024) uint8_t stage[kStages][kStage];
  Info info[kInfo];
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void mma_f16_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

using Cursor = KvCursor<kRows, kTokens>;

// A CTA's consecutive units of one item.
struct Run {
  Cursor c;
  int tiles;         // units of the run
  long long left;    // units of the CTA's share from the run's beginning on

  __device__ bool begins() const { return c.at == 0; }
  __device__ bool ends() const { return c.at + tiles == c.units; }
  // Whether the second tile has rows.
  __device__ bool second(const KvWork& w) const {
    return (long long)c.s.n * w.a.group - (long long)c.r * kRows > kRows / 2;
  }
  __device__ void open() { tiles = (int)min(left, (long long)(c.units - c.at)); }
  __device__ bool next(const KvWork& w) {
    left -= tiles;
    if (left <= 0) return false;
    c.next_item(w);
    open();
    return true;
  }
};

// The row of Q that a softmax thread owns: scaled by a power of two that puts its
// largest magnitude into [2^14, 2^15), where fp16 holds bfloat16 exactly down to 2^-24
// of it, and by the sign of the scale; into the thread's row of shared memory.
struct Row {
  float coef;    // scores: coef * 2^(byte - 127) * S
  int limit;     // tokens that the row sees; INT_MAX for a row that is not there
};
template <int D, bool kVec>
__device__ __forceinline__ Row load_row(const KvWork& w, const Cursor& c, int tile, int row, uint8_t* q) {
  const int rr = c.r * kRows + tile * 128 + row;
  const bool there = rr < c.s.n * w.a.group;
  Row out{1.f, INT_MAX};
  const uint32_t dst = smem_u32(q) + (uint32_t)row * 128u;
  const int swz = row & 7;
  if (!there) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) st_shared_v4(dst + (i >> 3) * 16384 + (((i & 7) ^ swz) << 4), 0, 0, 0, 0);
    return out;
  }
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(w.a.q) +
                             (long long)(c.s.start + rr / w.a.group) * w.a.q_row +
                             (long long)(c.h * w.a.group + rr % w.a.group) * w.a.q_head;
  uint32_t x[D / 2];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    if constexpr (kVec) {
      const uint4 u = reinterpret_cast<const uint4*>(src)[i];
      x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
    } else {
      const unsigned short* p = reinterpret_cast<const unsigned short*>(src) + 8 * i;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = p[2 * e] | ((uint32_t)p[2 * e + 1] << 16);
    }
  }
  uint32_t top = 0;   // magnitudes compare as integers; a NaN is above an infinity
#pragma unroll
  for (int i = 0; i < D / 2; ++i) top = max(top, max(x[i] << 16 & 0x7fff0000u, x[i] & 0x7fff0000u));
  const bool bad = top >= 0x7f800000u;
  const int e = min(max((int)(top >> 23), 27), 254);
  const float scale = w.a.scale;
  float up = __int_as_float((127 + 14 + 127 - e) << 23);
  if (scale < 0.f) up = -up;
  if (scale == 0.f) up = 0.f;
  if (scale != 0.f) out.coef = fabsf(scale) * 1.4426950408889634f * __int_as_float((e - 14) << 23);
  out.limit = kv_visible(c.s, rr / w.a.group, w.a.causal);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = x[4 * i + k];
      u[k] = bad ? 0x7e007e00u : half_pair(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
    }
    st_shared_v4(dst + (i >> 3) * 16384 + (((i & 7) ^ swz) << 4), u[0], u[1], u[2], u[3]);
  }
  return out;
}

template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tiles_kernel(const KvWork w) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  constexpr int kQTile = Smem<D>::kQTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.drained, 1);
    fence_mbarrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const uint32_t s_col[2] = {0, 128}, o_col[2] = {256, 384};
  chain_wait();

  // a wait whose outcome is the same for the whole warp
  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) -> bool {
    return __all_sync(~0u, mbar_wait(bar, parity, &sm.abort, w.a.err, site));
  };

  const long long total = kv_total_units<kRows, kTokens>(w);
  const long long share = max((total + w.ctas - 1) / w.ctas, (long long)kMinTiles);
  const long long begin = (long long)blockIdx.x * share;
  Run run;
  run.left = min(max(total - begin, 0ll), share);
  const bool work = run.left > 0;
  if (work) {
    run.c.seek(w, begin);
    run.open();
  }

  if (warp < 8) {
    // ---------------- softmax: a row a thread ----------------
    const int x = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;     // 32 lanes a warp, in bits 16 and up
    const uint32_t s_tmem = tmem + lanes + s_col[x], o_tmem = tmem + lanes + o_col[x];
    KvPart left[2] = {{0, 0, 0, kPartNone}, {0, 0, 0, kPartNone}};
    uint32_t s_phase = 0, o_phase = 0;
    int tile = 0;            // tiles of the CTA before the run
    bool more = work, ok = true;
    Row r{1.f, INT_MAX};
    auto put_row = [&] {
      if (x && !run.second(w)) return;
      r = load_row<D, kVec>(w, run.c, x, row, sm.q + x * kQTile);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[x]);
    };
    if (more) put_row();
    while (more && ok) {
      const Run now = run;
      const bool mine = !x || now.second(w);
      float m = kKvNone, l = 0.f;
      int vref = 0;
      const Row me = r;
      if (mine) {
        for (int j = 0; j < now.tiles; ++j) {
          if (!(ok = wait(&sm.s_full[x], s_phase, 0x501))) break;
          s_phase ^= 1;
          tc_fence_after();
          const Info& info = sm.info[(tile + j) % kInfo];
          const int cut = me.limit - (now.c.at + j) * kTokens;   // columns that the row sees
          const int missing = info.missing;
          const bool mask = __any_sync(~0u, cut < kTokens) || missing;
          uint32_t a[32], b[32];
          // columns of the half from `from` on that are masked, to -inf
          auto masked = [&](int from) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (from + i >= cut || (missing >> ((from + i) / kKvBlock) & 1)) a[i] = 0xff800000u;
              if (from + 32 + i >= cut || (missing >> ((from + 32 + i) / kKvBlock) & 1)) b[i] = 0xff800000u;
            }
          };
          auto factor = [&](int block) { return fmaxf(me.coef * info.kpow[block], 1.17549435e-38f); };
          auto top16 = [&](const uint32_t* v) {
            float t = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
            for (int i = 2; i < 16; i += 2) t = fmaxf(t, fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
            return t;
          };
          auto top_half = [&](int first) {
            return fmaxf(fmaxf(top16(a) * factor(first), top16(a + 16) * factor(first + 1)),
                         fmaxf(top16(b) * factor(first + 2), top16(b + 16) * factor(first + 3)));
          };
          tmem_ld32x2(s_tmem + 64, a, s_tmem + 96, b);
          if (mask) masked(64);
          float top = top_half(4);
          tmem_ld32x2(s_tmem, a, s_tmem + 32, b);
          if (mask) masked(0);
          top = fmaxf(top, top_half(0));
          const int vmax = info.vmax;
          if (__any_sync(~0u, top > m + kKvSlack) || vmax > vref) {
            const float up = fmaxf(m, top);
            float down = exp2_approx(m - up);
            m = up;
            l *= down;
            if (vmax > vref) {
              down *= exp2_approx((float)(vref - vmax));
              vref = vmax;
            }
            if (j > 0) {
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld32(o_tmem + i, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
                tmem_st32(o_tmem + i, o);
              }
            }
          }
          // 16 columns: P, packed in pairs, and its sum
          auto exp16 = [&](const uint32_t* v, int block, uint32_t* p) {
            const float f = factor(block);
            const int d = max(info.ve[block] - vref, -100);
            const float add = (float)d + kLift - m;
            const float2 f2 = make_float2(f, f), add2v = make_float2(add, add);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 y = fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, add2v);
              const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
              sum = add2(sum, e);
              p[i] = half_pair(e.x, e.y);
            }
            l += (sum.x + sum.y) * __int_as_float((127 - d) << 23);
          };
          auto exp_half = [&](int first, uint32_t p_tmem) {
            uint32_t p[32];
            exp16(a, first, p);
            exp16(a + 16, first + 1, p + 8);
            exp16(b, first + 2, p + 16);
            exp16(b + 16, first + 3, p + 24);
            tmem_st32_async(p_tmem, p);
          };
          exp_half(0, s_tmem);
          tmem_ld32x2(s_tmem + 64, a, s_tmem + 96, b);
          if (mask) masked(64);
          exp_half(4, s_tmem + 32);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[x]);
        }
      }
      tile += now.tiles;
      if (!ok) break;
      // the next run's rows, under the last products of this one
      more = run.next(w);
      if (more) put_row();
      const bool whole = now.begins() && now.ends();
      const int slot = now.begins() ? 1 : 0;
      if (!whole)
        left[slot] = KvPart{now.c.b, now.c.r, now.c.h,
                            kPartHeld | (now.begins() ? kPartBegins : 0) | (now.ends() ? kPartEnds : 0)};
      if (mine) {
        if (!(ok = wait(&sm.o_full[x], o_phase, 0x502))) break;
        o_phase ^= 1;
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float vscale = kv_power(vref);
        const int rr = now.c.r * kRows + x * 128 + row;
        const bool there = rr < now.c.s.n * w.a.group;
        __nv_bfloat16* dst = nullptr;
        float* into = nullptr;
        if (whole) {
          if (there) dst = static_cast<__nv_bfloat16*>(w.a.out) + kv_out_row(w.a, now.c.s, now.c.h, rr) * D;
        } else {
          into = reinterpret_cast<float*>(w.ws + (size_t)(2 * blockIdx.x + slot) * kv_part_bytes(D, kRows));
          reinterpret_cast<float2*>(into + kRows * D)[x * 128 + row] = make_float2(m, l);
          into += (x * 128 + row) * D;
        }
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          tmem_ld32(o_tmem + i, o);
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * inv * vscale;
          if (dst) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const float z[8] = {y[e], y[e + 1], y[e + 2], y[e + 3], y[e + 4], y[e + 5], y[e + 6], y[e + 7]};
              kv_store8(dst + i + e, z);
            }
          } else if (into) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(into + i + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        tc_fence_before();
      }
    }
    if (threadIdx.x < 2) w.parts[2 * blockIdx.x + threadIdx.x] = left[threadIdx.x];
  } else if (warp < 12) {
    // ---------------- keys and values: pages to fp16 operands ----------------
    const int c = threadIdx.x - 256;
    // a thread takes 16 bytes of a row; four neighbours and the same of the next token lie in different banks
    constexpr int kChunks = D / 16;                    // of a row
    constexpr int kPer = kChunks * kKvBlock / 128;     // rounds of 128 threads a block (2 blocks a round for D = 64)
    constexpr int kRounds = kBlocks * kChunks * kKvBlock / 128;
    const int chunk = (c & 3) + (kChunks == 8 ? (c >> 3 & 1) * 4 : 0);
    const int token0 = kChunks == 8 ? ((c >> 4) * 2 + (c >> 2 & 1)) : (c >> 2);   // of a round's 16 or 32
    constexpr int kRoundTokens = 128 / kChunks;
    static_assert(kPer <= 1, "a round holds whole blocks");
    const uint32_t dst0 = (uint32_t)(chunk >> 2) * 16384u + (uint32_t)token0 * 128u;
    const uint32_t piece = (uint32_t)(chunk & 3) * 2u, swz = (uint32_t)token0 & 7u;
    long long blocks = -1;      // lane i: place in the cache of block i of the tile that is fetched, -1: not there
    uint4 k[kRounds], v[kRounds];
    uint32_t stage = 0, phase = 1;
    int tile = 0;
    bool ok = true;

    // the tile's blocks, and their bytes for the softmax (by the first of the four warps)
    int ke = 0, ve = 0;
    auto find = [&](const Cursor& cur, int unit) {
      blocks = -1;
      if (lane < kBlocks) {
        const int blk = unit * kBlocks + lane;
        if ((long long)blk * kKvBlock < cur.s.seen) {
          const int page = __ldg(w.a.batch.table + (size_t)cur.b * w.a.batch.width + blk / w.a.cache.bpp);
          if (page >= 0 && page < w.a.cache.pages)
            blocks = ((long long)page * w.a.cache.heads + cur.h) * w.a.cache.bpp + blk % w.a.cache.bpp;
        }
        if (warp == 8 && blocks >= 0) {
          ke = __ldg(w.a.cache.ke + blocks);
          ve = __ldg(w.a.cache.ve + blocks);
        }
      }
    };
    auto fetch = [&](uint4 (&into)[kRounds], const int8_t* from) {
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const long long block = __shfl_sync(~0u, blocks, i * (kRoundTokens / kKvBlock) + token0 / kKvBlock);
        into[i] = block < 0 ? make_uint4(0, 0, 0, 0)
                            : ldg_nc_v4(from + block * (kKvBlock * D) + (token0 % kKvBlock) * D + chunk * 16);
      }
    };
    auto put = [&](const uint4 (&from)[kRounds]) -> bool {
      if (!wait(&sm.empty[stage], phase, 0x503)) return false;
      const uint32_t base = smem_u32(sm.stage[stage]) + dst0;
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const uint32_t u[4] = {from[i].x ^ 0x80808080u, from[i].y ^ 0x80808080u, from[i].z ^ 0x80808080u,
                               from[i].w ^ 0x80808080u};
        const uint32_t at = base + (uint32_t)(i * kRoundTokens) * 128u;
        st_shared_v4(at + ((piece ^ swz) << 4), bytes_low(u[0]), bytes_high(u[0]), bytes_low(u[1]), bytes_high(u[1]));
        st_shared_v4(at + (((piece + 1) ^ swz) << 4), bytes_low(u[2]), bytes_high(u[2]), bytes_low(u[3]),
                     bytes_high(u[3]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.full[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
      return true;
    };
    bool more = work;
    if (more) {
      find(run.c, run.c.at);
      fetch(k, w.a.cache.k);
    }
    while (more && ok) {
      const int tiles = run.tiles;
      for (int j = 0; j < tiles && ok; ++j, ++tile) {
        fetch(v, w.a.cache.v);
        if (warp == 8) {
          const unsigned absent = __ballot_sync(~0u, lane < kBlocks && blocks < 0);
          int vmax = blocks >= 0 ? ve : 0;
#pragma unroll
          for (int o = 4; o; o >>= 1) vmax = max(vmax, __shfl_xor_sync(~0u, vmax, o));
          Info& info = sm.info[tile % kInfo];
          if (lane < kBlocks) {
            info.kpow[lane] = blocks >= 0 ? kv_power(ke) : 0.f;
            info.ve[lane] = blocks >= 0 ? ve : vmax;
          }
          if (lane == 0) {
            info.vmax = vmax;
            info.missing = (int)absent;
          }
        }
        if (!(ok = put(k))) break;
        // the next tile's blocks and keys, before this one's values are put
        if (j + 1 < tiles) {
          find(run.c, run.c.at + j + 1);
          fetch(k, w.a.cache.k);
        } else if ((more = run.next(w))) {
          find(run.c, run.c.at);
          fetch(k, w.a.cache.k);
        }
        if (!(ok = put(v))) break;
      }
    }
  } else if (warp == 12) {
    // ---------------- one thread issues the MMAs ----------------
    if (lane == 0 && work) {
      constexpr uint32_t s_desc = idesc_f16_f32(128, kTokens, false, false);
      constexpr uint32_t o_desc = idesc_f16_f32(128, D, false, true);
      uint32_t stage = 0, phase = 0;       // of the ring
      uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
      bool ok = true, more = true;
      auto wait1 = [&](uint64_t* bar, uint32_t parity, unsigned site) {
        return mbar_wait(bar, parity, &sm.abort, w.a.err, site);
      };
      auto scores = [&](int x, uint32_t k_stage) {
        const uint32_t q = smem_u32(sm.q) + x * kQTile, k = smem_u32(sm.stage[k_stage]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t at = (uint32_t)(i >> 2) * 16384u + (uint32_t)(i & 3) * 32u;
          tc_mma_f16(tmem + s_col[x], sdesc_sw128(q + at, 16u, 1024u), sdesc_sw128(k + at, 16u, 1024u), s_desc, i > 0);
        }
        tc_commit(&sm.s_full[x]);
      };
      auto step = [&](uint32_t& st, uint32_t& ph) {
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      };
      while (more && ok) {
        const int heads = run.second(w) ? 2 : 1;   // row tiles
        uint32_t k_stage = stage;
        if (!(ok = wait1(&sm.full[stage], phase, 0x504))) break;
        step(stage, phase);
        for (int x = 0; x < heads && ok; ++x) {
          if (!(ok = wait1(&sm.q_full[x], q_phase[x], 0x505))) break;
          q_phase[x] ^= 1;
          tc_fence_after();
          scores(x, k_stage);
        }
        if (!ok) break;
        tc_commit(&sm.empty[k_stage]);
        for (int j = 0; j < run.tiles && ok; ++j) {
          const bool last = j + 1 == run.tiles;
          const uint32_t v_stage = stage;
          if (!(ok = wait1(&sm.full[stage], phase, 0x506))) break;
          step(stage, phase);
          for (int x = 0; x < heads; ++x) {
            if (!(ok = wait1(&sm.p_full[x], p_phase[x], 0x507))) break;
            p_phase[x] ^= 1;
            tc_fence_after();
            const uint32_t v = smem_u32(sm.stage[v_stage]);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
              mma_f16_tmem(tmem + o_col[x], tmem + s_col[x] + 8 * i, sdesc_sw128(v + 2048u * i, 16384u, 1024u), o_desc,
                           j > 0 || i > 0);
            if (last) {
              tc_commit(&sm.o_full[x]);
            } else {
              if (x == 0) {
                k_stage = stage;
                if (!(ok = wait1(&sm.full[stage], phase, 0x508))) break;
                step(stage, phase);
                tc_fence_after();
              }
              scores(x, k_stage);
            }
          }
          if (!ok) break;
          tc_commit(&sm.empty[v_stage]);
          if (!last) tc_commit(&sm.empty[k_stage]);
        }
        if (ok) more = run.next(w);
      }
      // what was issued has to end before tensor memory is given back
      tc_commit(&sm.drained);
      mbar_wait(&sm.drained, 0, nullptr, w.a.err, 0x509);
    }
    __syncwarp();
  }
  chain_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t tiles_sized(const KvWork& w, bool vec, cudaStream_t s) {
  auto kern = vec ? &kv_attention_tiles_kernel<D, true> : &kv_attention_tiles_kernel<D, false>;
  constexpr int bytes = (int)sizeof(Smem<D>);
  static_assert(bytes <= 227 * 1024, "one CTA an SM");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  e = launch_chained(kern, dim3(w.ctas), dim3(kThreads), bytes, 1, s, w);
  if (e != cudaSuccess) return e;
  return launch_chained(&kv_attention_join_kernel<D, kRows, __nv_bfloat16>, dim3(w.ctas, 8), dim3(256), 0, 1, s, w);
}

}  // namespace

size_t kv_tiles_workspace(int head_dim) { return (size_t)num_sms() * 2 * (sizeof(KvPart) + kv_part_bytes(head_dim, kRows)); }

cudaError_t launch_kv_attention_tiles(const KvAttentionArgs& a, long long rows_from, void* workspace, int head_dim,
                                      bool vec, cudaStream_t s) {
  KvWork w{};
  w.a = a;
  w.rows_from = rows_from;
  w.rows_to = LLONG_MAX;
  w.ctas = num_sms();
  if (w.ctas <= 0) return cudaErrorInvalidDevice;
  w.parts = static_cast<KvPart*>(workspace);
  w.ws = static_cast<uint8_t*>(workspace) + (size_t)w.ctas * 2 * sizeof(KvPart);
  return head_dim == 64 ? tiles_sized<64>(w, vec, s) : tiles_sized<128>(w, vec, s);
}

}  // namespace qmm
