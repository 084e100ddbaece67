// Attention over the 8-bit key-value cache for few rows: a token, or a few drafted
// ones, of each sequence.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp2(c q.k_j - m),   c = scale * log2(e)
//
// What bounds it is the cache: every byte of it is read once, and 2 * group * 2
// operations are made of each. So the work is cut by bytes. All (sequence, key head,
// tile of rows) items are laid end to end in blocks of 16 tokens, and every warp of
// the GPU takes the same number of consecutive blocks, wherever items begin and end:
// long and short sequences balance, and one long sequence spreads over all SMs. Where
// an item's blocks fall to several warps, the warps of a CTA join their parts through
// shared memory, and a second kernel joins what several CTAs hold, both in the order
// of the blocks.
//
// Inside a warp, tokens are the rows (M = 16: one block, one scale) and query rows the
// columns (N = 8) of mma m16n8k16 in fp16: S^T = K Q^T, O^T = V^T P^T. A group of up to
// 8 query heads then costs one MMA where rows of queries would pad to 16. int8 is exact
// in fp16. bfloat16 rows of Q are scaled by a power of two each, under which fp16
// holds them exactly down to 2^-24 of the row's largest value; float32 rows are split
// in two fp16 parts (22 bits), and so are their P. The order of a sum's terms is free,
// so a lane's 16 consecutive bytes of K serve four k-steps as they come, and its bytes
// of V are interleaved by token pairs. Each warp has a ring of blocks of its own, filled
// by cp.async 512 contiguous bytes at a time (where a lane copied just the bytes that it
// reads itself, in runs of 64 and 128, the long sequence took 68 us in place of 58).
//
// The running maximum moves only when some score is 8 (a factor of 256) above it, which a
// vote finds out. P is held times 2^6, at most 2^14, and fp16 ends 30 binades below that 2^6.
// V's powers of two go into V's own fp16 (the windows of kv_attention.cuh). A block outside
// of the window takes a path of its own, which ends when all rows are in one unit again:
// 64 sequences of 8192 tokens take 190 us with equal bytes or bytes within a window, 205 with
// bytes anywhere in 40 binades (float32 203 and 244).
//
// Measured, with the join: 64 sequences of up to 16384 tokens, 64 query heads on 8 of
// 128, 117 us (5.9 TB/s, 87 % of a copy; the copies without arithmetic took 114); one of
// 131072 54 us; one of 1021 9.7 us, a chain of latencies.
#include "kv_attention.cuh"

namespace qmm {

namespace {

constexpr int kLift = 6;             // P is held times 2^kLift
constexpr int kMinBlocks = 1;        // blocks a warp, at least

template <int D, int NT, int kWarps>
struct Shape {
  static constexpr int kRows = 8 * NT;
  // What fits beside the parts; 3 to 5 stages of D = 128 were the same within 1 %.
  static constexpr int kStages = D == 64 ? (kWarps == 8 ? 8 : 5) : kWarps == 12 ? 3 : NT == 1 ? 5 : 4;
  static constexpr int kChunk = 2 * kKvBlock * D;                 // K and V of one block
  static constexpr int kStage = kChunk + 128;                     // and a word a lane
  static constexpr int kRing = kStages * kStage;                  // a warp's
  static constexpr int kPartBytes = (int)kv_part_bytes(D, kRows);   // rows of O, then (m, l) each
  static_assert(kRing >= kPartBytes, "a warp's last part takes the place of its ring");
  static constexpr int kParts = kWarps * (kRing + kPartBytes);      // where the parts' descriptions are
  static constexpr int kState = kParts + 2 * kWarps * (int)sizeof(KvPart);
  static constexpr int kSmem = kState + kWarps * kRows * (int)sizeof(float2);
  static_assert(kSmem <= 227 * 1024, "one CTA an SM");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <int D, int NT, int kWarps, typename T, bool kVec>
__global__ void __launch_bounds__(32 * kWarps, 1) kv_attention_rows_kernel(const KvWork w) {
  using S = Shape<D, NT, kWarps>;
  constexpr bool kSplit = sizeof(T) == 4;   // float32: two fp16 parts
  constexpr int kParts = kSplit ? 2 : 1;
  constexpr int kKI = D / 64;               // 16-byte pieces of a K row a lane
  constexpr int kVW = D / 32;               // words of a V row a lane
  constexpr int kMT = D / 16;               // tiles of O^T
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* const ring = smem + warp * S::kRing;
  uint8_t* const first_part = smem + kWarps * S::kRing + warp * S::kPartBytes;
  KvPart* const parts = reinterpret_cast<KvPart*>(smem + S::kParts);
  float2* const state = reinterpret_cast<float2*>(smem + S::kState) + warp * S::kRows;   // of each row: below
  if (lane < 2) parts[2 * warp + lane] = KvPart{};
  chain_wait();

  const KvBatchArgs& batch = w.a.batch;
  const int heads = w.a.cache.heads, bpp = w.a.cache.bpp;

  KvCursor<S::kRows, kKvBlock, 0> at;   // of the block that is computed
  const int count = (int)at.open(w, w.ctas * kWarps, kMinBlocks, blockIdx.x * kWarps + warp);
  if (count > 0) {
    // What is fetched next is worked out 32 blocks at a time, a lane each, one window ahead: the table's entry, then
    // the block's place and its two bytes are loads that follow each other.
    KvCursor<S::kRows, kKvBlock, 0> ahead = at;   // of the first block in no window
    int planned = 0;
    int page = -1, within = 0, page_head = 0;     // the next window: the table's entry, the block in the page, the head
    auto plan = [&] {
      const int n = min(32, count - planned);
      page = -1;
      for (int k = 0; k < n;) {
        const int m = min(ahead.units - ahead.at, n - k), blk = ahead.at + lane - k;
        if (lane >= k && lane < k + m && (long long)blk * kKvBlock < ahead.s.seen) {
          const int p = (unsigned)blk / (unsigned)bpp;
          within = blk - p * bpp;
          page_head = ahead.h;
          page = __ldg(batch.table + (size_t)ahead.b * batch.width + p);
        }
        k += m;
        ahead.at += m;
        if (ahead.at == ahead.units && planned + k < count) ahead.next_item(w);
      }
      planned += n;
    };
    long long next_block = 0;
    uint32_t next_tag = 0;                        // 0: not there; else the two bytes, above them a 1
    auto locate = [&] {
      next_tag = 0;
      if (page >= 0 && page < w.a.cache.pages) {
        next_block = ((long long)page * heads + page_head) * bpp + within;
        next_tag = 0x10000u | __ldg(w.a.cache.ke + next_block) | ((uint32_t)__ldg(w.a.cache.ve + next_block) << 8);
      }
    };
    plan();
    long long block = 0;                          // the window that is fetched from
    uint32_t tag = 0;
    const uint32_t ring_addr = smem_u32(ring);
    // A block's K, then its V, lie in a stage as in memory, but for the 16-byte places of each 128 bytes, which are
    // exchanged so that neither the copies nor the loads below meet in a bank: by bits 1 and 2 ^ 0 of the row for
    // D = 128 (bits 1 and 2 of the place), by the pair of rows for D = 64 (the same bits).
    const uint32_t line = lane >> 3;   // of a copy's four
    const uint32_t copy_to = line * 128 + (((lane & 7) ^ (D == 128 ? (line & 2) | (line & 1) << 2 : line << 1)) << 4);
    const uint32_t k_from =
        D == 128 ? g * 128 + ((t ^ ((g & 2) | ((g >> 2 ^ g) & 1) << 2)) << 4)
                 : (g >> 1) * 128 + ((((g & 1) << 2 | t) ^ (g >> 1 & 3) << 1) << 4);
    const uint32_t v_from = D == 128 ? 2 * t * 128 + ((g ^ ((t & 1) << 1 | (t & 2) << 1)) << 4)
                                     : t * 128 + (((g >> 1) ^ t << 1) << 4) + (g & 1) * 8;

    auto fetch = [&](int index, int stage) {
      const int i = index & 31;
      if (i == 0) {
        block = next_block;
        tag = next_tag;
        if (planned < count) plan();
      }
      if (i == 16 && index + 16 < count) locate();
      const long long from = __shfl_sync(~0u, block, i) * (kKvBlock * D);
      const uint32_t what = __shfl_sync(~0u, tag, i);
      reinterpret_cast<uint32_t*>(ring + stage * S::kStage + S::kChunk)[lane] = what;
      if (what) {
        const uint32_t dst = ring_addr + stage * S::kStage + copy_to;
        const int8_t* const k = w.a.cache.k + from + lane * 16;
        const int8_t* const v = w.a.cache.v + from + lane * 16;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint32_t at = (D == 128 && (j & 1) ? dst ^ 64 : dst) + j * 512;
          cp_async16(at, k + j * 512);
          cp_async16(at + kKvBlock * D, v + j * 512);
        }
      }
      cp_commit();
    };
    int fetched = 0;

    uint32_t qf[kParts][NT][D / 16][2];
    float coef[NT][2];          // of columns 2t, 2t + 1
    int lim[NT][2];
    float m[NT][2], l[NT][2];
    float o[kMT][NT][4];
    int least = 0;
    // `settled`: all rows that have seen anything have O in the present window, and l in units of 2^m; else `state`
    // holds what the two are, (behind, window), for each row.
    int window = kKvNoWindow;
    bool settled = true;
    bool fresh = true, begins = at.at == 0;
    int stage = 0;
#pragma unroll 1
    for (int done = 0; done < count; ++done) {
      if (done == 0) {
        // the first blocks, ahead of the rows of Q
        locate();
#pragma unroll 1
        for (; fetched < S::kStages - 1; ++fetched) {
          if (fetched < count) fetch(fetched, fetched);
          else cp_commit();
        }
      }
      if (fresh) {
        fresh = false;
        // the item's rows: lane (g, t) holds elements 64 i + 16 t .. of row 8 nt + g
        least = INT_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int row = at.r * S::kRows + 8 * nt + g;
          const bool there = row < at.s.n * w.a.group;
          float x[kKI][2][8];
          float top = 0.f;
          const T* q = static_cast<const T*>(w.a.q) +
                       (there ? (long long)(at.s.start + row / w.a.group) * w.a.q_row +
                                    (long long)(at.h * w.a.group + row % w.a.group) * w.a.q_head
                              : 0);
#pragma unroll
          for (int i = 0; i < kKI; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (there) {
                kv_load8<kVec>(q + 64 * i + 16 * t + 8 * u, x[i][u]);
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][u][e] = 0.f;
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                // a NaN counts as an infinity here: fp16 then holds infinities, and the row's scores are not numbers
                top = fmaxf(top, x[i][u][e] == x[i][u][e] ? fabsf(x[i][u][e]) : __int_as_float(0x7f800000));
              }
            }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          // the largest magnitude to [2^14, 2^15)
          const int e = min(max(__float_as_int(top) >> 23, 27), 254);
          const float up = __int_as_float((127 + 14 + 127 - e) << 23);
          const bool bad = top > kKvMax;
          float cf = bad ? __int_as_float(0x7fc00000) : w.a.scale * 1.4426950408889634f * __int_as_float((e - 14) << 23);
#pragma unroll
          for (int i = 0; i < kKI; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int p2 = 0; p2 < 4; ++p2) {
                const float a0 = bad ? 0.f : x[i][u][2 * p2] * up, a1 = bad ? 0.f : x[i][u][2 * p2 + 1] * up;
                const uint32_t hi = half_pair(a0, a1);
                const int step = i * 4 + 2 * u + (p2 >> 1);
                qf[0][nt][step][p2 & 1] = hi;
                if constexpr (kSplit) qf[1][nt][step][p2 & 1] = half_rest(a0, a1, hi);
              }
          const int seen = there ? kv_visible(at.s, row / w.a.group, w.a.causal) : 0;
          least = min(least, there ? seen : INT_MAX);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            coef[nt][c] = __shfl_sync(~0u, cf, 4 * (2 * t + c));
            lim[nt][c] = __shfl_sync(~0u, seen, 4 * (2 * t + c));
            m[nt][c] = kKvNone;
            l[nt][c] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
        }
#pragma unroll
        for (int d = 16; d >= 4; d >>= 1) least = min(least, __shfl_xor_sync(~0u, least, d));
        window = kKvNoWindow;
        settled = true;
      }

      // fetch the block kStages - 1 ahead, over the one that all lanes have read, then wait for this one's copies
      __syncwarp();
      if (fetched < count) fetch(fetched, stage == 0 ? S::kStages - 1 : stage - 1);
      else cp_commit();
      ++fetched;
      cp_wait<S::kStages - 1>();
      __syncwarp();
      const uint32_t src = ring_addr + stage * S::kStage;
      const uint32_t word = reinterpret_cast<const uint32_t*>(ring + stage * S::kStage + S::kChunk)[lane];
      if (word) {
        // S^T
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[nt][c] = 0.f;
#pragma unroll
        for (int i = 0; i < kKI; ++i) {
          const uint32_t at = src + (i ? k_from ^ 64 : k_from);
          const uint4 k0 = ld_shared_v4(at), k1 = ld_shared_v4(at + 8 * D);
          const uint32_t r0[4] = {k0.x, k0.y, k0.z, k0.w}, r1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t u0 = r0[j] ^ 0x80808080u, u1 = r1[j] ^ 0x80808080u;
            const uint32_t a0 = bytes_low(u0), a1 = bytes_low(u1), a2 = bytes_high(u0), a3 = bytes_high(u1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int p = 0; p < kParts; ++p)
                mma16816(sc[nt], a0, a1, a2, a3, qf[p][nt][4 * i + j][0], qf[p][nt][4 * i + j][1]);
          }
        }
        const float kpow = kv_power(word & 255);
        const int ve = (word >> 8) & 255;
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float f = coef[nt][c] * kpow;
            if (fabsf(f) > kKvMax) f = copysignf(kKvMax, f);   // (0 times it is a score; a NaN stays one)
            sc[nt][c] *= f;
            sc[nt][c + 2] *= f;
          }
        const int token = at.at * kKvBlock + g;
        if (at.at * kKvBlock > least - kKvBlock) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (token + 8 * (c >> 1) >= lim[nt][c & 1]) sc[nt][c] = -INFINITY;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) over |= sc[nt][c] > m[nt][c & 1] + kKvSlack;
        const bool moved = !kv_in_window(ve, window, kKvBelow<T>);
        const bool first = window == kKvNoWindow;
        const int was = window;
        if (moved) window = kv_move_window(window, ve, ve, kKvBelow<T>);
        if (!first && (moved || !settled)) {
          bool now_settled = true;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(sc[nt][c], sc[nt][c + 2]), largest = 0.f;
#pragma unroll
              for (int i = 0; i < kMT; ++i) largest = fmaxf(largest, fmaxf(fabsf(o[i][nt][c]), fabsf(o[i][nt][c + 2])));
#pragma unroll
              for (int d = 16; d >= 4; d >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                largest = fmaxf(largest, __shfl_xor_sync(~0u, largest, d));
              }
              float2* const mine = state + 8 * nt + 2 * t + c;
              const float2 held = *mine;
              KvUnit u{m[nt][c], settled ? 0.f : held.x, settled ? was : __float_as_int(held.y)};
              const KvFactor f = kv_change_units(u, l[nt][c], top, largest, window);
              m[nt][c] = u.m;
#pragma unroll
              for (int i = 0; i < kMT; ++i) {
                o[i][nt][c] = o[i][nt][c] * f.a * f.b;
                o[i][nt][c + 2] = o[i][nt][c + 2] * f.a * f.b;
              }
              now_settled &= u.m == kKvNone || (u.window == window && u.behind == 0.f);
              sc[nt][c] += fmaxf(u.behind - kKvFar, 0.f);
              sc[nt][c + 2] += fmaxf(u.behind - kKvFar, 0.f);
              __syncwarp();   // the column's lanes have all read it
              *mine = make_float2(u.behind, __int_as_float(u.window));
            }
          settled = __all_sync(~0u, now_settled);
        } else if (__any_sync(~0u, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(sc[nt][c], sc[nt][c + 2]);
#pragma unroll
              for (int d = 16; d >= 4; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
              top = fmaxf(top, m[nt][c]);
              const float down = exp2_approx(m[nt][c] - top);
              m[nt][c] = top;
              l[nt][c] *= down;
#pragma unroll
              for (int i = 0; i < kMT; ++i) {
                o[i][nt][c] *= down;
                o[i][nt][c + 2] *= down;
              }
            }
        }
        uint32_t pf[kParts][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float sum[2] = {};
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = exp2_approx(sc[nt][2 * r] - m[nt][0]), p1 = exp2_approx(sc[nt][2 * r + 1] - m[nt][1]);
            sum[0] += p0;
            sum[1] += p1;
            const float w0 = p0 * (1 << kLift), w1 = p1 * (1 << kLift);
            const uint32_t hi = half_pair(w0, w1);
            pf[0][nt][r] = transpose8(hi);
            if constexpr (kSplit) pf[1][nt][r] = transpose8(half_rest(w0, w1, hi));
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            l[nt][c] += settled ? sum[c] : sum[c] * exp2_approx(fminf(state[8 * nt + 2 * t + c].x, kKvFar));
        }
        // O^T
        const KvScale vscale = kv_scale(ve - window);
        uint32_t vw[4][kVW];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // tokens 2t, 2t + 1, 2t + 8, 2t + 9
          const uint32_t at = src + kKvBlock * D + (j & 1 ? v_from ^ 64 : v_from) + (D == 128 ? (j & 1) * 128 : 0) +
                              (j >> 1) * 8 * D;
          if constexpr (D == 128) {
            const uint4 x = ld_shared_v4(at);
            vw[j][0] = x.x; vw[j][1] = x.y; vw[j][2] = x.z; vw[j][3] = x.w;
          } else {
            const uint2 x = ld_shared_v2(at);
            vw[j][0] = x.x; vw[j][1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < kVW; ++j) {
          // bytes of tokens (2t, 2t + 1) and (2t + 8, 2t + 9), side by side
          const uint32_t a = vw[0][j] ^ 0x80808080u, b = vw[1][j] ^ 0x80808080u;
          const uint32_t c = vw[2][j] ^ 0x80808080u, d = vw[3][j] ^ 0x80808080u;
          const uint32_t ab[2] = {prmt(a, b, 0x5140u), prmt(a, b, 0x7362u)};
          const uint32_t cd[2] = {prmt(c, d, 0x5140u), prmt(c, d, 0x7362u)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t a0 = bytes_low(ab[e], vscale), a1 = bytes_high(ab[e], vscale);
            const uint32_t a2 = bytes_low(cd[e], vscale), a3 = bytes_high(cd[e], vscale);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int p = 0; p < kParts; ++p)
                mma16816(o[2 * j + e][nt], a0, a1, a2, a3, pf[p][nt][0], pf[p][nt][1]);
          }
        }
      }
      if (++stage == S::kStages) stage = 0;

      // the end of the item, or of this warp's share of it
      const bool ends = at.at + 1 == at.units;
      if (ends || done + 1 == count) {
        uint8_t* into = nullptr;
        if (!(begins && ends)) {
          // a part: the one at the share's beginning to its own place, one at its end to the ring's, which
          // nothing is fetched to any more
          const int slot = done + 1 == count && begins ? 1 : 0;
          into = slot ? ring : first_part;
          if (slot) cp_wait<0>();
          __syncwarp();
          if (lane == 0)
            parts[2 * warp + slot] =
                KvPart{at.s.start, at.h, at.r * S::kRows, min(at.s.n * w.a.group - at.r * S::kRows, S::kRows),
                       kPartHeld | (begins ? kPartBegins : 0) | (ends ? kPartEnds : 0)};
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float sum = l[nt][c];
#pragma unroll
            for (int d = 16; d >= 4; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int col = 8 * nt + 2 * t + c;
            const float unlift = (into ? kKvPartScale : 1.f) / (1 << kLift);
            // O's power of two over that of l; by two factors where one might leave float32's range
            float unit = m[nt][c], scale = kv_power(window), again = 1.f;
            if (!settled) {
              const float2 held = state[col];
              unit -= held.x;
              scale = again = exp2f(0.5f * (held.x + (float)(__float_as_int(held.y) - 127)));
            }
            float y[kMT][2];
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
              y[i][0] = o[i][nt][c] * inv * unlift * scale * again;
              y[i][1] = o[i][nt][c + 2] * inv * unlift * scale * again;
            }
            if (into) {
              float* dst = reinterpret_cast<float*>(into) + col * D + g * (D / 8);
#pragma unroll
              for (int i = 0; i < kMT; i += 2)
                *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(y[i][0], y[i][1], y[i + 1][0], y[i + 1][1]);
              if (g == 0) reinterpret_cast<float2*>(into + S::kRows * D * 4)[col] = make_float2(unit, sum);
            } else {
              const int row = at.r * S::kRows + col;
              if (row < at.s.n * w.a.group) {
                T* dst = static_cast<T*>(w.a.out) + kv_out_row(w.a, at.s.start, at.h, row) * D + g * (D / 8);
#pragma unroll
                for (int i = 0; i < kMT; i += 4) {
                  const float z[8] = {y[i][0],     y[i][1],     y[i + 1][0], y[i + 1][1],
                                      y[i + 2][0], y[i + 2][1], y[i + 3][0], y[i + 3][1]};
                  kv_store8(dst + 2 * i, z);
                }
              }
            }
          }
        fresh = begins = true;
      }
      if (ends) at.next_item(w);
      else ++at.at;
    }
    cp_wait<0>();
  }

  // the parts of the CTA's warps, joined: every warp takes some of the rows
  __syncthreads();
  // runs of parts of one item: a run begins where a part begins its item, or with the first part
  const int flags = lane < 2 * kWarps ? parts[lane].flags : 0;
  unsigned held = __ballot_sync(~0u, flags & kPartHeld);
  const unsigned begin_mask = __ballot_sync(~0u, flags & kPartBegins), end_mask = __ballot_sync(~0u, flags & kPartEnds);
  KvPart left0{}, left1{};   // what goes to the workspace
  while (held) {
    const int first = __ffs(held) - 1;
    const unsigned later = held & begin_mask & ~((2u << first) - 1);
    const unsigned run = later ? held & ((later & (0u - later)) - 1) : held;   // the run's parts, a bit each
    held &= ~run;
    const KvPart a = parts[first];
    const bool begins = begin_mask >> first & 1, whole = begins && (end_mask & run);
    if (!whole) {
      KvPart& left = begins ? left1 : left0;
      left = a;
      left.flags = kPartHeld | (begins ? kPartBegins : 0) | (end_mask & run ? kPartEnds : 0);
    }
    // lane i: the place of the run's i-th part
    const int count_parts = __popc(run);
    int nth = 0, i = 0;
    for (unsigned m = run; m; m &= m - 1, ++i)
      if (lane == i) nth = __ffs(m) - 1;
    const uint32_t place = nth & 1 ? (nth >> 1) * S::kRing : kWarps * S::kRing + (nth >> 1) * S::kPartBytes;
    uint8_t* into = w.ws + (size_t)(2 * blockIdx.x + (begins ? 1 : 0)) * kv_part_bytes(D, S::kRows);
    for (int row = warp; row < a.rows; row += kWarps) {
      T* out = nullptr;
      if (whole) out = static_cast<T*>(w.a.out) + kv_out_row(w.a, a.start, a.h, a.first + row) * D;
      kv_join_row<D, T>(count_parts, S::kRows, row, [&](int j) { return smem + __shfl_sync(~0u, place, j); }, whole, out,
                        into);
    }
  }
  if (threadIdx.x == 0) {
    w.parts[2 * blockIdx.x] = left0;
    w.parts[2 * blockIdx.x + 1] = left1;
  }
  chain_release();
}

// Two tiles of eight rows where one tile would not hold a sequence's rows.
int row_tiles(int group, int max_tokens) { return (long long)group * max_tokens <= 8 ? 1 : 2; }

// Which kernels a call needs. Sequences with up to few_rows rows a key head are this
// file's, those with more the tensor cores' (tcgen05): a tile there is 128 rows, filled
// or not, and one of float32, alone on its SM, takes as long as about two of the rows
// kernel's of 16 (8 tokens of 4 heads over 32000 there, 12 here: 51 us both). For
// bfloat16 two tiles of 16 rows are slower on long caches (64 sequences of up to 16384
// with 24 rows each: 277 us, 247 there), if faster on short ones (one of 1021: 13 us, 23):
// a choice by rows alone, because lengths are on the device.
// A call whose sequences all have max_tokens rows needs one kernel.
int few_rows(bool bf16) { return bf16 ? 16 : 32; }
struct Plan {
  bool few, many;
  size_t few_bytes, bytes;   // the workspace: `few` first
};
Plan plan_of(int rows, int batch, int group, int head_dim, int max_tokens, bool bf16) {
  Plan p{};
  p.many = (long long)group * max_tokens > few_rows(bf16);
  p.few = !p.many || (long long)max_tokens * batch != rows;
  const int part_rows = p.many ? 16 : 8 * row_tiles(group, max_tokens);
  if (p.few) p.few_bytes = (size_t)num_sms() * 2 * (sizeof(KvPart) + kv_part_bytes(head_dim, part_rows));
  p.bytes = p.few_bytes + (p.many ? kv_tiles_workspace(head_dim, bf16) : 0);
  return p;
}

template <int D, int NT, int kWarps, typename T>
cudaError_t rows_launch(const KvWork& w, bool vec, bool join, cudaStream_t s) {
  using S = Shape<D, NT, kWarps>;
  constexpr auto kVector = &kv_attention_rows_kernel<D, NT, kWarps, T, true>;
  constexpr auto kScalar = &kv_attention_rows_kernel<D, NT, kWarps, T, false>;
  cudaError_t e = vec ? kv_allow_smem<kVector>(S::kSmem) : kv_allow_smem<kScalar>(S::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_chained(vec ? kVector : kScalar, dim3(w.ctas), dim3(32 * kWarps), S::kSmem, 1, s, w);
  if (e != cudaSuccess || !join) return e;
  return launch_chained(&kv_attention_join_kernel<D, S::kRows, T>, dim3(w.ctas), dim3(256), 0, 1, s, w);
}

template <int D, int NT, typename T>
cudaError_t rows_typed(const KvAttentionArgs& a, bool with_tiles, bool vec, cudaStream_t s, KvWork& w) {
  const int sms = num_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  w.a = a;
  w.rows_to = with_tiles ? few_rows(sizeof(T) == 2) : LLONG_MAX;
  w.parts = static_cast<KvPart*>(a.workspace);
  w.ws = static_cast<uint8_t*>(a.workspace) + (size_t)sms * 2 * sizeof(KvPart);
  // one CTA an SM, but no more than the work can fill, as far as the table's width says
  const long long tiles = ((long long)a.batch.rows * a.group + 8 * NT - 1) / (8 * NT) + a.batch.batch;
  const long long blocks = std::max(1, (a.batch.capacity + kKvBlock - 1) / kKvBlock);
  const long long bound = std::min(tiles * a.cache.heads, 1ll << 30) * blocks;
  auto ctas = [&](int warps) { return (int)std::min<long long>(sms, (bound + warps * kMinBlocks - 1) / (warps * kMinBlocks)); };
  // Twelve warps, which hide more of the arithmetic behind the copies (64 sequences of up to 16384 tokens 127 -> 117
  // us in bfloat16, 150 -> 122 in float32), but eight where there are few blocks a warp to hide it behind (one
  // sequence of 1021 tokens 10.9 -> 9.9 us), and for 16 rows, whose accumulators leave no registers for twelve (156
  // -> 151 us).
  if constexpr (NT == 1) {
    if (bound > 2ll * 8 * sms) {
      w.ctas = ctas(12);
      return rows_launch<D, NT, 12, T>(w, vec, !with_tiles, s);
    }
  }
  w.ctas = ctas(8);
  return rows_launch<D, NT, 8, T>(w, vec, !with_tiles, s);
}

template <int D>
cudaError_t rows_sized(const KvAttentionArgs& a, bool with_tiles, bool bf16, bool vec, cudaStream_t s, KvWork& w) {
  if (!with_tiles && row_tiles(a.group, a.max_tokens) == 1)
    return bf16 ? rows_typed<D, 1, __nv_bfloat16>(a, false, vec, s, w) : rows_typed<D, 1, float>(a, false, vec, s, w);
  return bf16 ? rows_typed<D, 2, __nv_bfloat16>(a, with_tiles, vec, s, w) : rows_typed<D, 2, float>(a, with_tiles, vec, s, w);
}

}  // namespace

size_t kv_attention_workspace(int rows, int batch, int heads, int group, int head_dim, int max_tokens, bool bf16) {
  return plan_of(rows, batch, group, head_dim, max_tokens, bf16).bytes;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int head_dim, bool bf16, bool vec, cudaStream_t s,
                                const char** kernel_name) {
  const Plan p = plan_of(a.batch.rows, a.batch.batch, a.group, head_dim, a.max_tokens, bf16);
  KvWork few{};
  if (p.few) {
    const cudaError_t e = head_dim == 64 ? rows_sized<64>(a, p.many, bf16, vec, s, few)
                                         : rows_sized<128>(a, p.many, bf16, vec, s, few);
    if (e != cudaSuccess) return e;
    *kernel_name = "kv_attention_rows";
  }
  if (p.many) {
    const cudaError_t e = launch_kv_attention_tiles(a, p.few ? &few : nullptr,
                                                    static_cast<uint8_t*>(a.workspace) + p.few_bytes, head_dim, bf16,
                                                    vec, s);
    if (e != cudaSuccess) return e;
    *kernel_name = p.few ? "kv_attention_rows+tiles" : "kv_attention_tiles";
  }
  return cudaSuccess;
}

}  // namespace qmm
