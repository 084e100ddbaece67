// Attention over the 8-bit key-value cache for many rows: prompts, pieces of them, an
// encoder's states, on the tensor cores (tcgen05).
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
// other runs. Its roles: warps 0-3 and 4-7 hold a row a thread (its maximum and sum need
// no exchange); one warp copies int8 keys and values from their pages (bulk copies of a
// block each), warps 8-11 widen them to fp16, exactly, into a ring of three operands;
// one warp issues the MMAs, another works out the CTA's share of the work. A key block's
// power of two goes into the factor of its 16 columns of S, a value block's into its fp16
// (the windows of kv_attention.cuh). A tile with blocks that no one window holds is passed
// several times, each time for the blocks of one window. The running maximum moves only
// past a score 8 above it (rescaling O is then rare); scores are masked only in tiles that
// some row's limit cuts.
//
// The work is cut like that of the other kernel (kv_attention.cuh), a unit being a tile
// of 128 tokens, so that short and long rows of causal prompts balance.
//
// Float32 queries take one tile of 128 rows: Q in two fp16 parts (22 bits) fills both
// tiles' places, P in two parts all the columns of S, and either product runs twice.
//
// Measured: a prompt of 8192 tokens, 32 query heads on 8 of 128, 435 us (1264 TFLOP/s),
// float32 1255 us; 8192 x 8192 not causal 772 us (1424); 500 tokens over 32000 200 us
// (1300). A tile of 256 x 128 takes about 3200 cycles: its MMAs 2080, its traffic in shared
// memory (320 KB: Q and K 128, V 64, copies and conversion 128) 2560, one tile's softmax
// 1500. Sixteen softmax warps with half a row each, and taking half of P before the maximum
// is known, were slower (853 and 889 us where this took 798). Windows: a prompt of 4096 143
// us with equal bytes, 145 with bytes within a window, 203 with a block of zeros in a
// hundred, 492 with bytes anywhere in 40 binades (float32 369, 369, 442, 1608).
#include "kv_attention.cuh"

namespace qmm {
namespace {

constexpr int kTokens = 128;
// Rows of an item: two tiles of 128, or one of float32, whose two fp16 parts take the
// places of both.
template <typename T>
constexpr int kTileRows = sizeof(T) == 4 ? 128 : 256;
constexpr int kThreads = 512;
// Registers a thread of the softmax, of the converters and of the rest: the launch has 128 each.
constexpr int kSoftmaxRegs = 192, kConvertRegs = 80, kRestRegs = 48;
static_assert(256 * kSoftmaxRegs + 128 * kConvertRegs + 128 * kRestRegs <= 512 * 128, "registers of the launch");
constexpr int kStages = 3;                 // operands (K or V tiles) in the ring of fp16
constexpr int kRaw = 4;                    // and in the ring of int8 before it
constexpr int kInfo = 4;                   // passes whose scales are kept
constexpr int kBlocks = kTokens / kKvBlock;
// Units that stand for what an item costs beside its tiles. Chosen on a prompt of bfloat16 and 128 columns; 64 columns
// and float32, whose items and tiles cost others, have not been measured for it.
constexpr int kSetup = 5;
constexpr int kMinUnits = kSetup + 2;      // a CTA's share, at least
constexpr float kLift = 7.f;               // P is held times 2^7: at most 2^15
// Sums of D <= 128 products of fp16 below 2^15 and int8 are below 2^29: with factors up to this scores stay below 2^20,
// where the rounding of one is 2^-4 at most.
constexpr float kPlainFactor = 1.f / 512;

// A pass over a tile, as the softmax, the converters and the MMAs' warp need to know it.
struct alignas(16) Info {
  float kpow[kBlocks];     // 2^(byte - 127) of the key blocks
  KvScale v[kBlocks];      // the value blocks' powers of two over the window's
  int window;
  int missing;             // blocks on pages that are not there, or of other passes, a bit each
  int first;               // the tile's first token
  int last;                // the last pass of the run
  float kmax;              // of kpow
  int pad[3];
};

// A CTA's consecutive units of one item, as one warp works them out for all.
struct alignas(16) Run {
  int b, r, h, flags;          // as in a part; kRunStop: there is none
  int at, tiles, rows, start;  // first unit, units, rows of the tile pair, first packed row
  int n, len, seen;            // the sequence's
  int slot;                    // of this record
};
enum { kRunStop = 8 };
constexpr int kRuns = 4;       // kept

// What bounds the waits, in shared memory: read only where one is long.
struct Watch {
  uint64_t limit, raw_limit;   // ns; of the wait at kSiteRaw
  int abort;
};
template <int D>
struct Smem {
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kStage = kTokens * D * 2;
  static constexpr int kRawStage = kTokens * D;
  alignas(1024) uint8_t q[2 * kQTile];
  alignas(1024) uint8_t stage[kStages][kStage];
  alignas(128) uint8_t raw[kRaw][kRawStage];
  Info info[kInfo];
  Run run[kRuns];
  int run_pass[kRuns];     // the number of each run's first pass
  KvScale plain[kBlocks];  // 1, for K
  uint64_t full[kStages], empty[kStages], raw_full[kRaw], raw_empty[kRaw];
  uint64_t run_full[kRuns], run_empty[kRuns];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], drained;   // p_full: of either half of the columns
  uint32_t tmem;
  Watch watch;
};

// MMAs by the one lane of a converged warp for which `lead` is not 0: predicated, so
// that the warp's descriptors stay in uniform registers, where the instruction takes
// them from. A from shared memory, then A from tensor memory.
__device__ __forceinline__ void mma_one(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_one(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "sub.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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

// A wait of a whole warp, whose outcome is the same for all its lanes. Bounded by the
// clock like the other kernels', which is read, with the abort flag, only every kLook
// tries: the waits here are many and mostly shorter than the reading. (A role may wait for
// as long as one item takes, about 14 ms a million tokens.)
constexpr uint32_t kLook = 256;
enum { kSiteRaw = 0x503 };   // the converters' wait for int8 keys or values
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile Watch* watch, unsigned* err,
                                         unsigned site) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    if (i % kLook == 0) {
      if (__any_sync(~0u, watch->abort != 0)) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(~0u, now - t0 > (site == kSiteRaw ? watch->raw_limit : watch->limit))) {
        record_error(err, site);
        watch->abort = 1;
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 128 columns of this warp's lanes.
__device__ __forceinline__ void tmem_ld128(uint32_t t, uint32_t (&r)[128]) {
  auto& a = *reinterpret_cast<uint32_t(*)[32]>(&r[0]);
  auto& b = *reinterpret_cast<uint32_t(*)[32]>(&r[32]);
  auto& c = *reinterpret_cast<uint32_t(*)[32]>(&r[64]);
  auto& d = *reinterpret_cast<uint32_t(*)[32]>(&r[96]);
  tmem_ld32x2(t, a, t + 32, b);
  tmem_ld32x2(t + 64, c, t + 96, d);
}

// Where rows of a tile lie, in steps: row rr is query head rr % group of token rr / group,
// of a tensor with `row` elements between tokens and `head` between heads.
struct Walk {
  long long at;            // elements from the sequence's first row and the key head's first query head
  long long step, wrap;    // a step, and what is added where it passes a token's last head
  int head, heads, group;
  __device__ Walk(int rr, int rows, int g, long long row, long long head_stride) : group(g) {
    const int token = (unsigned)rr / (unsigned)g, tokens = (unsigned)rows / (unsigned)g;
    head = rr - token * g;
    heads = rows - tokens * g;
    at = token * row + head * head_stride;
    step = tokens * row + heads * head_stride;
    wrap = row - g * head_stride;
  }
  __device__ void next() {
    head += heads;
    at += step;
    if (head >= group) {
      head -= group;
      at += wrap;
    }
  }
};

// The rows of Q of a softmax warp's 32 threads, a row each. They come with neighbouring
// lanes on neighbouring 16 bytes (a lane a row would ask for 32 lines at a time, and
// take 8000 cycles of the L1 cache for the CTA's 64 KB), straight into the operand's
// rows (`q`: the warp's first), and are converted there: scaled by a power of two each
// that puts a row's largest magnitude into [2^14, 2^15), where fp16 holds bfloat16
// exactly down to 2^-24 of it, and by the sign of the scale.
struct Row {
  float coef;    // scores: coef * 2^(byte - 127) * S
  int limit;     // tokens that the row sees; INT_MAX for a row that is not there
};
template <int D, typename T, bool kVec>
__device__ __forceinline__ Row load_rows(const KvWork& w, const Run& run, int first, uint32_t q) {
  constexpr int kRows = kTileRows<T>;
  const int lane = threadIdx.x & 31;
  if constexpr (sizeof(T) == 4) {
    // Float32: the first half of a row comes into its place in one operand, the second half into that in the other;
    // what they become, the row's two fp16 parts, is held until both have been read.
    constexpr uint32_t kOther = 128 * D * 2;
    constexpr int kHalf = D / 8, kLanes = 2 * kHalf, kAtOnce = 32 / kLanes;   // pieces of half a row, of a row; rows
    const int piece = lane % kLanes;
    {
      int row = lane / kLanes;
      Walk walk(run.r * kRows + first + row, kAtOnce, w.a.group, w.a.q_row, w.a.q_head);
      const float* src = static_cast<const float*>(w.a.q) + (long long)run.start * w.a.q_row +
                         (long long)run.h * w.a.group * w.a.q_head + piece * 4;
      const int within = piece % kHalf;
      const uint32_t to = q + (uint32_t)(piece / kHalf) * kOther + (uint32_t)(within >> 3) * 16384u;
#pragma unroll 4
      for (int i = 0; i < 32 / kAtOnce; ++i, row += kAtOnce, walk.next()) {
        const uint32_t dst = to + (uint32_t)row * 128u + (((within & 7) ^ (row & 7)) << 4);
        const float* at = src + walk.at;
        if (first + row >= run.rows) {
          st_shared_v4(dst, 0, 0, 0, 0);
        } else if constexpr (kVec) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(at) : "memory");
        } else {
          st_shared_v4(dst, __float_as_uint(at[0]), __float_as_uint(at[1]), __float_as_uint(at[2]), __float_as_uint(at[3]));
        }
      }
      if constexpr (kVec) asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
    const uint32_t mine = q + (uint32_t)lane * 128u, swz = (uint32_t)(lane & 7) << 4;
    auto place = [&](int i) {   // piece i of the row in one operand
      return mine + (uint32_t)(i >> 3) * 16384u + (((uint32_t)(i & 7) << 4) ^ swz);
    };
    auto from = [&](int i) { return place(i % kHalf) + (i >= kHalf ? kOther : 0u); };   // of the row as it came
    uint32_t top = 0;   // magnitudes compare as integers; a NaN is above an infinity
#pragma unroll 4
    for (int i = 0; i < kLanes; ++i) {
      const uint4 x = ld_shared_v4(from(i));
      top = max(max(max(top, x.x & 0x7fffffffu), max(x.y & 0x7fffffffu, x.z & 0x7fffffffu)), x.w & 0x7fffffffu);
    }
    const bool bad = top >= 0x7f800000u;
    const int e = min(max((int)(top >> 23), 27), 254);
    const float scale = w.a.scale;
    float up = __int_as_float((127 + 14 + 127 - e) << 23);
    up = scale < 0.f ? -up : scale == 0.f ? 0.f : up;
    uint32_t hi[D / 2], lo[D / 2];
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      const uint4 x = ld_shared_v4(from(i));
      const float y[4] = {__uint_as_float(x.x) * up, __uint_as_float(x.y) * up, __uint_as_float(x.z) * up,
                          __uint_as_float(x.w) * up};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        hi[2 * i + k] = bad ? 0x7e007e00u : half_pair(y[2 * k], y[2 * k + 1]);
        lo[2 * i + k] = bad ? 0u : half_rest(y[2 * k], y[2 * k + 1], hi[2 * i + k]);
      }
    }
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      st_shared_v4(place(i), hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
      st_shared_v4(place(i) + kOther, lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
    }
    Row out{0.f, INT_MAX};
    if (scale != 0.f) out.coef = fabsf(scale) * 1.4426950408889634f * __int_as_float((e - 14) << 23);
    if (first + lane < run.rows)
      out.limit = kv_visible(KvSeq{0, run.n, run.len, run.seen},
                             (unsigned)(run.r * kRows + first + lane) / (unsigned)w.a.group, w.a.causal);
    return out;
  } else {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;   // of a row; rows
  const int piece = lane % kLanes;
  {
    int row = lane / kLanes;
    Walk walk(run.r * kRows + first + row, kAtOnce, w.a.group, w.a.q_row, w.a.q_head);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(w.a.q) + (long long)run.start * w.a.q_row +
                               (long long)run.h * w.a.group * w.a.q_head + piece * 8;
#pragma unroll 4
    for (int i = 0; i < 32 / kAtOnce; ++i, row += kAtOnce, walk.next()) {
      const uint32_t dst = q + (uint32_t)(piece >> 3) * 16384u + (uint32_t)row * 128u + (((piece & 7) ^ (row & 7)) << 4);
      const __nv_bfloat16* at = src + walk.at;
      if (first + row >= run.rows) {
        st_shared_v4(dst, 0, 0, 0, 0);
      } else if constexpr (kVec) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(at) : "memory");
      } else {
        const unsigned short* p = reinterpret_cast<const unsigned short*>(at);
        st_shared_v4(dst, p[0] | ((uint32_t)p[1] << 16), p[2] | ((uint32_t)p[3] << 16), p[4] | ((uint32_t)p[5] << 16),
                     p[6] | ((uint32_t)p[7] << 16));
      }
    }
    if constexpr (kVec) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
  const uint32_t mine = q + (uint32_t)lane * 128u, swz = (uint32_t)(lane & 7) << 4;
  auto place = [&](int i) { return mine + (uint32_t)(i >> 3) * 16384u + (((uint32_t)(i & 7) << 4) ^ swz); };
  uint32_t tops = 0;   // magnitudes compare as integers, two at a time; a NaN is above an infinity
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 x = ld_shared_v4(place(i));
    tops = __vmaxu2(__vmaxu2(tops, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu)),
                    __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  }
  const uint32_t top = max(tops & 0xffffu, tops >> 16) << 16;
  const bool bad = top >= 0x7f800000u;
  const int e = min(max((int)(top >> 23), 27), 254);
  const float scale = w.a.scale;
  float up = __int_as_float((127 + 14 + 127 - e) << 23);
  up = scale < 0.f ? -up : scale == 0.f ? 0.f : up;
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 x = ld_shared_v4(place(i));
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = bad ? 0x7e007e00u : half_pair(__uint_as_float(u[k] << 16) * up, __uint_as_float(u[k] & 0xffff0000u) * up);
    st_shared_v4(place(i), y[0], y[1], y[2], y[3]);
  }
  Row out{0.f, INT_MAX};
  if (scale != 0.f) out.coef = fabsf(scale) * 1.4426950408889634f * __int_as_float((e - 14) << 23);
  if (first + lane < run.rows)
    out.limit = kv_visible(KvSeq{0, run.n, run.len, run.seen},
                           (unsigned)(run.r * kRows + first + lane) / (unsigned)w.a.group, w.a.causal);
  return out;
  }
}

template <int D, typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tiles_kernel(const KvWork w) {
  constexpr int kRows = kTileRows<T>;
  constexpr bool kSplit = sizeof(T) == 4;   // float32: Q and P in two fp16 parts each
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  constexpr int kQTile = Smem<D>::kQTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    const bool test = w.a.wait_ns && blockIdx.x == 0;
    sm.watch = Watch{test ? 4 * w.a.wait_ns : kWaitLimitNs, test ? w.a.wait_ns : kWaitLimitNs, 0};
    for (int i = 0; i < kBlocks; ++i) sm.plain[i] = kv_scale(0);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 4);
    }
    for (int i = 0; i < kRuns; ++i) {
      mbar_init(&sm.run_full[i], 1);
      mbar_init(&sm.run_empty[i], 14);   // 8 warps of the softmax, 4 converters, the MMAs' and the copies'
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
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
  chain_wait();

  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) -> bool {
    return wait_for(bar, parity, &sm.watch, w.a.err, site);
  };
  // the CTA's runs in turn
  int run_slot = 0;
  uint32_t run_phase = 0;
  auto next_run = [&](Run& to) -> bool {
    if (!wait(&sm.run_full[run_slot], run_phase, 0x50a)) return false;
    to = sm.run[run_slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.run_empty[run_slot]);
    if (++run_slot == kRuns) {
      run_slot = 0;
      run_phase ^= 1;
    }
    return !(to.flags & kRunStop);
  };

  if (warp < 8) {
    // ---------------- softmax: a row a thread ----------------
    more_registers<kSoftmaxRegs>();
    const int x = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;     // 32 lanes a warp, in bits 16 and up
    // scores (and P) of the two tiles in columns 0 and 128, O in 256 and 384
    const uint32_t s_tmem = tmem + lanes + x * 128, o_tmem = s_tmem + 256;
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    // the run, which stays in its place until it is done with: this role has no registers for it
    const Run* now = nullptr;
    auto hold_run = [&]() -> bool {
      if (!wait(&sm.run_full[run_slot], run_phase, 0x50a)) return false;
      now = &sm.run[run_slot];
      if (++run_slot == kRuns) {
        run_slot = 0;
        run_phase ^= 1;
      }
      return !(now->flags & kRunStop);
    };
    Row me{0.f, INT_MAX};
    const int first = x * 128 + (warp & 3) * 32;   // the warp's first row
    const uint32_t q_rows = smem_u32(sm.q) + x * kQTile + (warp & 3) * 32 * 128;
    auto put_rows = [&] {
      me = load_rows<D, T, kVec>(w, *now, first, q_rows);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[x]);
    };
    if (threadIdx.x == 0) w.parts[2 * blockIdx.x] = w.parts[2 * blockIdx.x + 1] = KvPart{};
    bool more = hold_run();
    if (more && (!x || now->rows > 128)) put_rows();
    while (more) {
      const bool mine = !x || now->rows > 128;
      KvUnit unit{kKvNone, 0.f, kKvNoWindow};
      float l = 0.f, above = -kKvMax;   // a score above it moves the maximum
      if (mine) {
        const float coef = me.coef;
        int pass = 0, last = 0;
        for (int j = 0; !last; ++j, ++pass) {
          if (!(ok = wait(&sm.s_full[x], s_phase, 0x501))) break;
          s_phase ^= 1;
          tc_fence_after();
          if (j == 0) pass = sm.run_pass[now->slot];
          const Info& info = sm.info[pass % kInfo];
          uint32_t s[128];
          tmem_ld128(s_tmem, s);
          const int missing = info.missing, window = info.window;
          const int cut = me.limit - info.first;   // columns of the tile that the row sees
          last = info.last;
          float by = coef, origin = 0.f;           // origin: what has been taken off the scores
          auto factor = [&](int k) { return fmaxf(by * info.kpow[k], 1.17549435e-38f); };
          const bool masked = cut < kTokens || missing, large = coef * info.kmax > kPlainFactor;
          if (__any_sync(~0u, masked || large)) {
            if (__any_sync(~0u, large)) {
              // Scores may be so large that what their rounding leaves out of the maximum, and the sum below would bring
              // back, is too much for P: they are counted from the largest of them, which makes that one 0. (Where they
              // lie, in a short loop: done in registers, it took the prompt of 8192 from 435 to 500 us without being
              // reached. The kernel's loops are as long as the instruction cache holds; the converters' is cut for it.)
              by = fminf(by, kKvMax / info.kmax);
              float most = -kKvMax;
#pragma unroll 1
              for (int k = 0; k < 2 * kBlocks; ++k) {
                uint32_t r[kKvBlock];
                const int block = k % kBlocks, seen = missing >> block & 1 ? 0 : cut - kKvBlock * block;
                tmem_ld16(s_tmem + kKvBlock * block, r);
                const float f = factor(block);
                if (k < kBlocks) {
#pragma unroll
                  for (int i = 0; i < kKvBlock; ++i)
                    if (i < seen) most = fmaxf(most, __uint_as_float(r[i]) * f);
                } else {
                  const float inverse = 1.f / f;
#pragma unroll
                  for (int i = 0; i < kKvBlock; ++i)
                    r[i] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(r[i]), f), most) * inverse);
                  tmem_st16(s_tmem + kKvBlock * block, r);
                }
              }
              origin = most;
              tmem_ld128(s_tmem, s);
            }
#pragma unroll
            for (int i = 0; i < kTokens; ++i)
              if (i >= cut || (missing >> (i / kKvBlock) & 1)) s[i] = 0xff800000u;
          }
          // the blocks' factors, and the largest score
          float f[kBlocks], top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kBlocks; ++k) {
            f[k] = factor(k);
            float t = __uint_as_float(s[16 * k]);
#pragma unroll
            for (int i = 1; i < 15; i += 2)
              t = fmaxf(fmaxf(t, __uint_as_float(s[16 * k + i])), __uint_as_float(s[16 * k + i + 1]));
            t = fmaxf(t, __uint_as_float(s[16 * k + 15]));
            top = fmaxf(top, t * f[k]);
          }
          top += origin;
          if (__any_sync(~0u, top > above || window != unit.window)) {
            float largest = 0.f;
            if (j > 0 && __any_sync(~0u, unit.m != kKvNone && top > -INFINITY && unit.window != window)) {
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                uint32_t o[16];
                tmem_ld16(o_tmem + i, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) largest = fmaxf(largest, fabsf(__uint_as_float(o[e])));
              }
            }
            const KvFactor by_units = kv_change_units(unit, l, top, largest, window);
            above = unit.m - fmaxf(unit.behind, 0.f) + kKvSlack;
            if (j > 0) {
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                uint32_t o[16];
                tmem_ld16(o_tmem + i, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by_units.a * by_units.b);
                tmem_st16(o_tmem + i, o);
              }
            }
          }
          // P = exp2(score - m), held times 2^kLift, and its sum (a row far above its scores: see kKvFar)
          const float behind = fminf(unit.behind, kKvFar);
          const float base = kLift - (unit.m - (unit.behind - behind) - origin);
          float sum = 0.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t p[32], rest[kSplit ? 32 : 1];
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k) {
              const float2 f2 = make_float2(f[k], f[k]), a2 = make_float2(base, base);
              float2 part = make_float2(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 y = fma2(
                    make_float2(__uint_as_float(s[16 * k + 2 * i]), __uint_as_float(s[16 * k + 2 * i + 1])), f2, a2);
                const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                part = i ? add2(part, e) : e;
                p[8 * (k & 3) + i] = half_pair(e.x, e.y);
                if constexpr (kSplit) {
                  const float2 of = __half22float2(*reinterpret_cast<const __half2*>(&p[8 * (k & 3) + i]));
                  const float2 left = sub2(e, of);
                  rest[8 * (k & 3) + i] = half_pair(left.x, left.y);
                }
              }
              sum += part.x + part.y;
            }
            tmem_st32_async(s_tmem + 32 * half, p);
            if constexpr (kSplit) tmem_st32_async(s_tmem + 64 + 32 * half, rest);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[x][half]);
          }
          l = fmaf(sum, exp2_approx(behind), l);
        }
      }
      if (!ok) break;
      const Run& was = *now;
      more = hold_run();
      const bool whole = (was.flags & kPartBegins) && (was.flags & kPartEnds);
      const int slot = was.flags & kPartBegins ? 1 : 0;
      if (!whole && threadIdx.x == 0)
        w.parts[2 * blockIdx.x + slot] = KvPart{was.start, was.h, was.r * kRows, was.rows, was.flags};
      if (mine) {
        if (!(ok = wait(&sm.o_full[x], o_phase, 0x502))) break;
        o_phase ^= 1;
        tc_fence_after();
        // O by way of this warp's rows of Q, whose last use is over, so that neighbouring lanes write neighbouring
        // bytes: 256 bytes of each row at a time, as bfloat16 or, of a part, as float32
        // 1 / l and O's power of two over that of l in one factor where that is a normal number, else in three
        const float inv = l == 0.f ? 0.f : (whole ? 1.f : kKvPartScale) / l;
        const float vscale = exp2f(0.5f * (unit.behind + (float)(unit.window - 127)));
        const float both = unit.behind == 0.f ? inv * kv_power(unit.window) : 0.f;
        const bool small = __any_sync(~0u, both < 1.17549435e-38f);
        const float2 factor = small ? make_float2(inv, inv) : make_float2(both, both);
        uint8_t* const part = w.ws + (size_t)(2 * blockIdx.x + slot) * kv_part_bytes(D, kRows);
        if (!whole) reinterpret_cast<float2*>(part + kRows * D * 4)[first + lane] = make_float2(unit.m - unit.behind, l);
        const bool narrow = whole && !kSplit;              // to bfloat16
        const int step = narrow ? D : D / 2;               // columns at a time: 2 D bytes of a row
        constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;   // pieces of 16 bytes of them; rows
        const int piece = lane % kPieces;
        const uint32_t mine_at = q_rows + (uint32_t)lane * 128u, swz = (uint32_t)(lane & 7) << 4;
#pragma unroll 1
        for (int col = 0; col < D; col += step) {
#pragma unroll 1
          for (int i = 0; i < step; i += 32) {
            uint32_t o[32];
            tmem_ld32(o_tmem + col + i, o);
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 v = mul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), factor);
              y[e] = v.x;
              y[e + 1] = v.y;
            }
            if (small) {
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = y[e] * vscale * vscale;
            }
            // piece p of the row: panel p / 8, place p % 8 exchanged by the row
            auto put = [&](int p, uint32_t u0, uint32_t u1, uint32_t u2, uint32_t u3) {
              st_shared_v4(mine_at + (uint32_t)(p >> 3) * 16384u + (((uint32_t)(p & 7) << 4) ^ swz), u0, u1, u2, u3);
            };
            if (narrow) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const __nv_bfloat162 h = __floats2bfloat162_rn(y[e + 2 * k], y[e + 2 * k + 1]);
                  u[k] = *reinterpret_cast<const uint32_t*>(&h);
                }
                put((i + e) / 8, u[0], u[1], u[2], u[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                put((i + e) / 4, __float_as_uint(y[e]), __float_as_uint(y[e + 1]), __float_as_uint(y[e + 2]),
                    __float_as_uint(y[e + 3]));
            }
          }
          __syncwarp();
          int row = lane / kPieces;
          // in bytes; a part's rows follow each other
          const long long out_heads = (long long)w.a.cache.heads * w.a.group;
          constexpr int kHead = D * (int)sizeof(T);
          Walk walk(was.r * kRows + first + row, kAtOnce, w.a.group, out_heads * kHead, kHead);
          uint8_t* to = static_cast<uint8_t*>(w.a.out) + (was.start * out_heads + was.h * w.a.group) * kHead +
                        (narrow ? 0 : 4 * col) + piece * 16;
          if (!whole) {
            walk = Walk(first + row, kAtOnce, 1, 4 * D, 0);
            to = part + 4 * col + piece * 16;
          }
#pragma unroll 4
          for (int i = 0; i < 32 / kAtOnce; ++i, row += kAtOnce, walk.next()) {
            const uint4 v = ld_shared_v4(q_rows + (uint32_t)(piece >> 3) * 16384u + (uint32_t)row * 128u +
                                         (((piece & 7) ^ (row & 7)) << 4));
            if (first + row < was.rows) *reinterpret_cast<uint4*>(to + walk.at) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.run_empty[was.slot]);
      if (more && (!x || now->rows > 128)) put_rows();
    }
  } else if (warp < 12) {
    // ---------------- int8 to fp16 operands ----------------
    fewer_registers<kConvertRegs>();
    const int c = threadIdx.x - 256;
    // A thread takes 16 bytes of a token's row. Of eight neighbours four read the first half of one token and
    // four the second half of the next (D = 128), so that neither their loads nor their swizzled stores meet
    // in a bank.
    constexpr int kChunks = D / 16;                    // of a row
    constexpr int kRoundTokens = 128 / kChunks;
    constexpr int kRounds = kTokens / kRoundTokens;
    const int odd = c >> 2 & 1;
    const int chunk = (c & 3) + (kChunks == 8 ? ((c >> 3 & 1) ^ odd) * 4 : 0);
    const int token0 = kChunks == 8 ? (c >> 4) * 2 + odd : c >> 2;
    const uint32_t src0 = (uint32_t)(token0 * D + chunk * 16);
    const uint32_t dst0 = (uint32_t)(chunk >> 2) * 16384u + (uint32_t)token0 * 128u;
    const uint32_t piece = (uint32_t)(chunk & 3) * 2u, swz = (uint32_t)token0 & 7u;
    const uint32_t at0 = dst0 + ((piece ^ swz) << 4), at1 = dst0 + (((piece + 1) ^ swz) << 4);
    uint32_t stage = 0, phase = 1, from = 0, from_phase = 0;
    bool ok = true;
    Run run{};
    int pass = 0, last = 0;
    bool value = false;   // K and V in turn
    while (ok && next_run(run)) {
#pragma unroll 1
      do {
        if (!(ok = wait(&sm.raw_full[from], from_phase, kSiteRaw))) break;
        const Info& info = sm.info[pass % kInfo];
        last = info.last;
        const KvScale* scales = (value ? info.v : sm.plain) + token0 / kKvBlock;
        uint32_t src = smem_u32(sm.raw[from]) + src0, dst = smem_u32(sm.stage[stage]);
#pragma unroll 1
        for (int r0 = 0; r0 < kRounds; r0 += 4) {
          uint4 x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = ld_shared_v4(src + r * (kRoundTokens * D));
          if (r0 == 0 && !(ok = wait(&sm.empty[stage], phase, 0x50c))) break;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t u[4] = {x[r].x ^ 0x80808080u, x[r].y ^ 0x80808080u, x[r].z ^ 0x80808080u,
                                   x[r].w ^ 0x80808080u};
            const uint32_t at = dst + (uint32_t)(r * kRoundTokens) * 128u;
            const KvScale k = scales[r * (kRoundTokens / kKvBlock)];
            st_shared_v4(at + at0, bytes_low(u[0], k), bytes_high(u[0], k), bytes_low(u[1], k), bytes_high(u[1], k));
            st_shared_v4(at + at1, bytes_low(u[2], k), bytes_high(u[2], k), bytes_low(u[3], k), bytes_high(u[3], k));
          }
          src += 4 * kRoundTokens * D;
          dst += 4 * kRoundTokens * 128u;
          scales += 4 * (kRoundTokens / kKvBlock);
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.full[stage]);
          mbar_arrive(&sm.raw_empty[from]);
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
        if (++from == kRaw) {
          from = 0;
          from_phase ^= 1;
        }
        pass += value;
        value = !value;
      } while (value || !last);
    }
  } else {
    fewer_registers<kRestRegs>();
    if (warp == 12) {
      // ---------------- the MMAs, by one lane of a converged warp ----------------
      constexpr uint32_t s_desc = idesc_f16_f32(128, kTokens, false, false);
      constexpr uint32_t o_desc = idesc_f16_f32(128, D, false, true);
      const uint32_t lead = elect();
      const uint32_t tm = __shfl_sync(~0u, tmem, 0);
      // descriptors of the first k-step; the others' differ in the start address alone, the low word
      const uint64_t q_first = sdesc_sw128(smem_u32(sm.q), 16u, 1024u);
      const uint64_t k_first = sdesc_sw128(smem_u32(sm.stage[0]), 16u, 1024u);
      const uint64_t v_first = sdesc_sw128(smem_u32(sm.stage[0]), 16384u, 1024u);
      uint32_t stage = 0, phase = 0;       // of the ring
      uint32_t q_phase = 0, p_phase = 0;   // a bit for either tile
      bool ok = true;
      // the next operand of the ring, waited for
      auto operand = [&](unsigned site) -> uint32_t {
        const uint32_t got = stage;
        ok = wait(&sm.full[got], phase, site);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
        return got;
      };
      Run run{};
      int pass = 0;
      while (ok && next_run(run)) {
        const int pair = __shfl_sync(~0u, run.rows, 0) > 128 ? 2 : 1;
        // scores of pass 0; then, pass by pass, the products of one and the scores of the next
        uint32_t v_stage = 0;
        bool more = true;
#pragma unroll 1
        for (int j = -1; more && ok; ++j) {
          uint32_t k_stage = 0;
          if (j >= 0) {
            v_stage = operand(0x506);
            more = !__shfl_sync(~0u, sm.info[pass++ % kInfo].last, 0);
          }
#pragma unroll 1
          for (int x = 0; x < pair && ok; ++x) {
            if (j >= 0) {
              const uint64_t v = v_first + v_stage * (Smem<D>::kStage / 16);
              const uint32_t o = tm + 256u + (uint32_t)x * 128u, p = tm + (uint32_t)x * 128u;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                if (!(ok = wait(&sm.p_full[x][half], p_phase >> x & 1, 0x507))) break;
                tc_fence_after();
#pragma unroll
                for (int i = half * (kBlocks / 2); i < (half + 1) * (kBlocks / 2); ++i)
                  mma_one(lead, o, p + 8 * i, v + 128u * i, o_desc, j > 0 || i > 0);
                if constexpr (kSplit) {
#pragma unroll
                  for (int i = half * (kBlocks / 2); i < (half + 1) * (kBlocks / 2); ++i)
                    mma_one(lead, o, p + 64 + 8 * i, v + 128u * i, o_desc, 1);
                }
              }
              if (!ok) break;
              p_phase ^= 1u << x;
              if (!more) commit_one(lead, &sm.o_full[x]);
            } else {
              if (!(ok = wait(&sm.q_full[x], q_phase >> x & 1, 0x505))) break;
              q_phase ^= 1u << x;
            }
            if (more) {
              if (x == 0) {
                k_stage = operand(0x508);
                if (!ok) break;
              }
              tc_fence_after();
              const uint64_t q = q_first + (uint32_t)x * (kQTile / 16), k = k_first + k_stage * (Smem<D>::kStage / 16);
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint32_t step = (uint32_t)((i >> 2) * 16384 + (i & 3) * 32) / 16;
                mma_one(lead, tm + (uint32_t)x * 128u, q + step, k + step, s_desc, i > 0);
                if constexpr (kSplit) mma_one(lead, tm, q + kQTile / 16 + step, k + step, s_desc, 1);
              }
              commit_one(lead, &sm.s_full[x]);
            }
          }
          if (!ok) break;
          if (j >= 0) commit_one(lead, &sm.empty[v_stage]);
          if (more) commit_one(lead, &sm.empty[k_stage]);
        }
      }
      // what was issued has to end before tensor memory is given back
      commit_one(lead, &sm.drained);
      mbar_wait(&sm.drained, 0, nullptr, w.a.err, 0x509);
      __syncwarp();
    } else if (warp == 14) {
      // ---------------- int8 keys and values from their pages, and what the softmax needs of their blocks ----------
      uint32_t stage = 0, phase = 1, copies = 0;
      int pass = 0;
      bool ok = true;
      Run run{};
      while (ok && next_run(run)) {
        int window = kKvNoWindow;
        bool opens = true;   // the run's first pass
        // four tiles at a time, a lane each block: the table and the scales are two loads that follow each other
#pragma unroll 1
        for (int j0 = 0; j0 < run.tiles && ok; j0 += 32 / kBlocks) {
          const int blk = (run.at + j0) * kBlocks + lane;
          long long block = -1;
          int ke = 0, ve = 0;
          if (j0 + lane / kBlocks < run.tiles && (long long)blk * kKvBlock < run.seen) {
            const int page = __ldg(w.a.batch.table + (size_t)run.b * w.a.batch.width + blk / w.a.cache.bpp);
            if (page >= 0 && page < w.a.cache.pages) {
              block = ((long long)page * w.a.cache.heads + run.h) * w.a.cache.bpp + blk % w.a.cache.bpp;
              ke = __ldg(w.a.cache.ke + block);
              ve = __ldg(w.a.cache.ve + block);
            }
          }
          const unsigned there = __ballot_sync(~0u, block >= 0);
#pragma unroll 1
          for (int j = j0; j < min(j0 + 32 / kBlocks, run.tiles) && ok; ++j) {
            unsigned pending = there & (((1u << kBlocks) - 1) << ((j - j0) * kBlocks));   // the tile's lanes
            do {
              unsigned here = __ballot_sync(~0u, kv_in_window(ve, window, kKvBelow<T>)) & pending;
              if (here != pending) {
                const bool open = pending >> lane & 1;
                const int lo = __reduce_min_sync(~0u, open ? ve : INT_MAX), hi = __reduce_max_sync(~0u, open ? ve : 0);
                constexpr int kWidth = kKvBelow<T> + kKvAbove;
                if (hi - lo <= kWidth || !here) {
                  window = kv_move_window(window, lo, min(hi, lo + kWidth), kKvBelow<T>);
                  here = __ballot_sync(~0u, kv_in_window(ve, window, kKvBelow<T>)) & pending;
                }
              }
              pending &= ~here;
              const bool mine = here >> lane & 1;
#pragma unroll 1
              for (int kind = 0; kind < 2; ++kind) {
                if (!(ok = wait(&sm.raw_empty[stage], phase, 0x50d))) break;
                if (kind == 0 && lane / kBlocks == j - j0) {
                  Info& info = sm.info[pass % kInfo];
                  const int i = lane % kBlocks;
                  const float power = mine ? kv_power(ke) : 0.f;
                  float most = power;
#pragma unroll
                  for (int o = kBlocks / 2; o; o >>= 1)
                    most = fmaxf(most, __shfl_xor_sync(((1u << kBlocks) - 1) << (lane & ~(kBlocks - 1)), most, o));
                  info.kpow[i] = power;
                  info.v[i] = kv_scale(mine ? ve - window : 0);
                  if (i == 0) {
                    info.kmax = most;
                    info.window = window;
                    info.missing = (int)(~here >> ((j - j0) * kBlocks) & ((1u << kBlocks) - 1));
                    info.first = (run.at + j) * kTokens;
                    info.last = !pending && j + 1 == run.tiles;
                    if (opens) sm.run_pass[run.slot] = pass;
                  }
                }
                __syncwarp();
                const bool drop = w.a.wait_ns && blockIdx.x == 0 && copies == 0;   // (the test of the waits)
                if (lane == 0 && !drop)
                  mbar_arrive_expect_tx(&sm.raw_full[stage], (uint32_t)__popc(here) * (kKvBlock * D));
                __syncwarp();
                if (mine && !drop)
                  bulk_load(smem_u32(sm.raw[stage]) + (lane % kBlocks) * (kKvBlock * D),
                            (kind ? w.a.cache.v : w.a.cache.k) + block * (kKvBlock * D), kKvBlock * D,
                            &sm.raw_full[stage]);
                ++copies;
                if (++stage == kRaw) {
                  stage = 0;
                  phase ^= 1;
                }
              }
              ++pass;
              opens = false;
            } while (pending && ok);
          }
        }
      }
      // copies in flight end before the CTA does, whatever ended the loop
      for (uint32_t i = copies > kRaw ? copies - kRaw : w.a.wait_ns && blockIdx.x == 0; i < copies; ++i)
        mbar_wait(&sm.raw_full[i % kRaw], (i / kRaw) & 1, nullptr, w.a.err, 0x50e);
      __syncwarp();
    } else if (warp == 13) {
      // ---------------- the CTA's share of the work, run by run ----------------
      KvCursor<kRows, kTokens, kSetup> c{};
      long long left = c.open(w, w.ctas, kMinUnits, blockIdx.x);
      uint32_t slot = 0, phase = 1;
      for (;;) {
        // the tiles of this stretch of units, if it has any
        const int units = left > 0 ? (int)min(left, (long long)(c.units - c.at)) : 0;
        const int from = max(c.at - kSetup, 0), tiles = max(c.at + units - kSetup, 0) - from;
        const bool end = left <= 0;
        if (end || tiles > 0) {
          if (!wait(&sm.run_empty[slot], phase, 0x50b)) break;
          if (lane == 0) {
            Run run{};
            run.flags = kRunStop;
            if (!end) {
              run = Run{c.b, c.r, c.h,
                        kPartHeld | (from == 0 ? kPartBegins : 0) | (c.at + units == c.units ? kPartEnds : 0), from, tiles,
                        min(c.s.n * w.a.group - c.r * kRows, kRows), c.s.start, c.s.n, c.s.len, c.s.seen, (int)slot};
            }
            sm.run[slot] = run;
            mbar_arrive(&sm.run_full[slot]);
          }
          __syncwarp();
          if (++slot == kRuns) {
            slot = 0;
            phase ^= 1;
          }
          if (end) break;
        }
        left -= units;
        if (left > 0) c.next_item(w);
      }
    }
  }
  chain_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D, typename T>
cudaError_t tiles_sized(const KvWork& w, const KvWork* few, bool vec, cudaStream_t s) {
  constexpr auto kVector = &kv_attention_tiles_kernel<D, T, true>, kScalar = &kv_attention_tiles_kernel<D, T, false>;
  constexpr int bytes = (int)sizeof(Smem<D>), kRows = kTileRows<T>, kSlices = 16;
  static_assert(bytes <= 227 * 1024, "one CTA an SM");
  cudaError_t e = vec ? kv_allow_smem<kVector>(bytes) : kv_allow_smem<kScalar>(bytes);
  if (e != cudaSuccess) return e;
  e = launch_chained(vec ? kVector : kScalar, dim3(w.ctas), dim3(kThreads), bytes, 1, s, w);
  if (e != cudaSuccess) return e;
  if (few)
    return launch_chained(&kv_attention_join_both_kernel<D, 16, kRows, T>, dim3(w.ctas, kSlices + 1), dim3(256), 0, 1, s,
                          *few, w);
  return launch_chained(&kv_attention_join_kernel<D, kRows, T>, dim3(w.ctas, kSlices), dim3(256), 0, 1, s, w);
}

}  // namespace

size_t kv_tiles_workspace(int head_dim, bool bf16) {
  return (size_t)num_sms() * 2 * (sizeof(KvPart) + kv_part_bytes(head_dim, bf16 ? kTileRows<__nv_bfloat16> : kTileRows<float>));
}

cudaError_t launch_kv_attention_tiles(const KvAttentionArgs& a, const KvWork* few, void* workspace, int head_dim, bool bf16,
                                      bool vec, cudaStream_t s) {
  KvWork w{};
  w.a = a;
  w.rows_from = few ? few->rows_to + 1 : 0;
  w.rows_to = LLONG_MAX;
  w.ctas = num_sms();
  if (w.ctas <= 0) return cudaErrorInvalidDevice;
  w.parts = static_cast<KvPart*>(workspace);
  w.ws = static_cast<uint8_t*>(workspace) + (size_t)w.ctas * 2 * sizeof(KvPart);
  if (head_dim == 64)
    return bf16 ? tiles_sized<64, __nv_bfloat16>(w, few, vec, s) : tiles_sized<64, float>(w, few, vec, s);
  return bf16 ? tiles_sized<128, __nv_bfloat16>(w, few, vec, s) : tiles_sized<128, float>(w, few, vec, s);
}

}  // namespace qmm
