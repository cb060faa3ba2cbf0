// q4nx_attention_block.cu -- attention of many query rows (prompt blocks) over
// the 4-bit cache, on the tcgen05 tensor cores.
//
//   S = q k^T (256 rows x 64 tokens),  p = exp2(S * scale * log2 e - ref),
//   O += p v,  l += sum p;  out = O / l
// with one running reference per row, moved only when a logit passes it by 2^8.
//
// Where the kernel for few rows keeps the codes exact and applies the groups'
// scales to the sums, here a key or value x = (code - 8) * scale + mid enters as
// two bf16 numbers, x = hi + lo within 2^-17 of itself (one alone, 2^-9, would
// move the row's log-sum by more than binary32 does), and so does p:
//   S = q k_hi + q k_lo          (q is bf16)
//   O = p_hi v_hi + p_lo v_hi + p_hi v_lo
// 28 tcgen05.mma (M = 128, K = 16) per 128 rows and 64 tokens at 128 channels,
// accumulated in binary32 in TMEM.
//
// Twenty warps, one CTA per SM: a loader (bulk copies of the cache's blocks), the
// MMA issuer, eight softmax warps (a thread is a row: its logits come from TMEM,
// its p take their place there, as the A operand of the second product) and eight
// decoding warps (codes to bf16 pairs in shared memory, 128-byte swizzle: keys as
// rows of channels, values as rows of tokens; two buffers each).  A unit is two
// tiles of 128 rows that share what is decoded: while the softmax of one is under
// way, the products of the other are.  With one tile per CTA (S in two buffers)
// decoding was half the work: 70 us instead of 52 for 64 tokens x 32 heads over
// 16384 positions, 8 kv heads of 128 channels, 30 us of it in the loop (14 steps).
//
// Bound: the turns that a tile takes in a step of 2.1 us: softmax 1.0, the issue and
// run of its products 0.9, the hand-over 0.2.  The products alone need 1.1 us for
// both tiles (tensor pipe 37% busy), and the warps issue 0.6 instructions a cycle
// and scheduler, so that neither is full: the next thing would be S in two buffers
// beside two tiles, for which TMEM (512 columns) has no room with q in it.  The
// start takes 8.6 us: plan, the first blocks' arrival, cold code.
// What else was tried: two issuing warps, one for each tile: they fall into step
// and leave the tensor cores idle together, 58 us instead of 52; the keys' wait
// before the weights': 53; both products as rolled loops: 55.
//
// A CTA's steps (64 tokens) are a range of all units' steps; a unit cut between
// CTAs leaves its parts in the workspace, with a record of whose they are, for
// a second kernel that joins them over the whole GPU (a part is 128 KB).
#include <cuda_fp16.h>

#include "q4nx_attention.cuh"

namespace q4nx {

namespace {

constexpr int kTile = 128, kRows = 2 * kTile;                   // rows of a tile (TMEM lanes), of a unit
constexpr int kSB = 4, kTok = kSB * kKvBlock;                   // blocks and tokens of a step
constexpr int kThreads = 640, kDecodeWarps = 8, kRawStages = 4;
constexpr int kWarpLoad = 0, kWarpMma = 1, kWarpSoft0 = 4, kWarpDecode0 = 12;
// registers per thread: 96 at launch, shared out anew (4, 8 and 8 warps)
constexpr int kRegsRest = 64, kRegsSoft = 144, kRegsDecode = 64;
static_assert(4 * kRegsRest + 8 * kRegsSoft + 8 * kRegsDecode <= kThreads / 32 * 96, "the split draws on the launch's registers");
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Layout {
  static constexpr int NBX = D / 64;
  static constexpr int kKeys = 2 * NBX * 8192;                  // hi boxes (64 tokens x 64 channels), then lo
  static constexpr int kValues = 2 * D * 128;                   // hi rows (D x 64 tokens), then lo
  static constexpr int kRaw = kSB * kv_block_bytes(D);
  static constexpr int kValuesAt = 2 * kKeys, kRawAt = kValuesAt + 2 * kValues, kControlAt = kRawAt + kRawStages * kRaw;
  // TMEM columns of a tile; p takes the place of S, 32 columns (32 tokens) at a time: 16 of p_hi, 16 of p_lo
  static constexpr uint32_t kQ = 0, kS = D / 2, kO = kS + kTok, kCols = kTmemCols / 2;
  static_assert(kO + D <= kCols, "TMEM budget");
  static_assert(kControlAt % 128 == 0 && kValuesAt % 1024 == 0, "swizzled regions");
};

struct Control {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_ready[2], s_full[2], p_full[2], o_full[2];  // of a tile
  uint64_t drain;
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
  volatile int odd_any[2];                          // the last step (from 1 on) with a value kept as NaN, by stage
  volatile int odd[2][4][kTok];                     // that of a group's token
  int64_t begin, end;
  int64_t prefix[kKvMaxBatch + 1], cost[kKvMaxBatch + 1];
};
template <int D>
constexpr int kSmemBytes = Layout<D>::kControlAt + sizeof(Control) + 1024;

// ---- PTX ----
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// K-major operand, 128-byte swizzle: rows of 128 B, 8-row groups 1024 B apart
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | static_cast<uint64_t>(1) << 16 | static_cast<uint64_t>(1024 >> 4) << 32 |
         static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// D fp32, A (TMEM) and B (shared memory) bf16, both K-major, M = 128, N = n
__host__ __device__ constexpr uint32_t idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((kTile >> 4) << 24);
}
// four products of K = 16 (A at columns a, a + A1, .., 128 bytes of B's rows),
// issued by one elected lane of a converged warp
template <uint32_t kId, int A1, int A2, int A3>
__device__ __forceinline__ void mma64(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 ra;\n\t.reg .b64 rb;\n\t"
      "setp.ne.b32 p, %3, 0;\n\tsetp.eq.b32 t, 1, 1;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
      "add.u32 ra, %1, %5;\n\tadd.u64 rb, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ra], rb, %4, t;\n\t"
      "add.u32 ra, %1, %6;\n\tadd.u64 rb, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ra], rb, %4, t;\n\t"
      "add.u32 ra, %1, %7;\n\tadd.u64 rb, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ra], rb, %4, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(accumulate), "n"(kId), "n"(A1), "n"(A2), "n"(A3)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// completes the loads before it: their registers pass through, so that no use is moved ahead of the wait
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
// with its wait
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t at, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }

// Bounded wait that also ends when another warp has given up; for a whole warp.
// The first wait sleeps without a look at the timer, whose read would lie between
// the phase's end and the warp's next step.
__device__ __forceinline__ bool wait(Control& c, uint64_t* bar, uint32_t parity, uint32_t* err) {
  bool ok = mbar_try_wait_sleep(bar, parity, 20000u);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    while (!(ok = mbar_try_wait_sleep(bar, parity, 1000000u))) {
      if (c.abort_flag) break;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        c.abort_flag = 1;
        atomicOr(err, kErrTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The positions that some row of a unit sees, [first, last], and those of its rows.
struct Span {
  int64_t first, last;
  int rows;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Unit& u, int from, int most) {     // its rows from .. from + most - 1
  Span s;
  const int64_t base = u.rq.L - u.rq.T, row0 = u.rg * kRows + from, left = u.rq.T * a.group - row0;
  s.rows = static_cast<int>(left < most ? left : most);
  if (s.rows <= 0) return {0, -1, 0};
  const int64_t p0 = base + quot(row0, a.group), p1 = base + quot(row0 + s.rows - 1, a.group);
  s.first = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
  s.last = p1 < u.rq.L ? p1 : u.rq.L - 1;
  return s;
}

// A CTA's range, piece by piece (a piece: its part of one unit), the same for
// every warp: steps that no row sees are left out by all of them.
struct Range {
  int lo, hi;
};
struct Walk {
  Unit u;
  Span s;
  int at, end;              // the CTA's steps of the piece
  int64_t step0;            // the request's step of the CTA's step 0
  Range r;                  // those that some row sees
};
__device__ __forceinline__ Range range_of(const Walk& w, const Span& s) {
  if (s.last < s.first) return {w.at, w.at};
  const int64_t lo = s.first / kTok - w.step0, hi = s.last / kTok + 1 - w.step0;
  const Range r = {lo > w.at ? static_cast<int>(lo < w.end ? lo : w.end) : w.at, hi < w.end ? static_cast<int>(hi > w.at ? hi : w.at) : w.end};
  return r;
}
__device__ __forceinline__ void next_piece(const AttnArgs& a, const Plan& pl, const Control& c, Walk& w, int steps) {
  w.at = w.end;
  w.u = find_unit<kSB, kRows>(a, pl, c.begin + w.at);
  w.s = span_of(a, w.u, 0, kRows);
  const int64_t end = w.u.start + w.u.n - c.begin;
  w.end = static_cast<int>(end < steps ? end : steps);
  w.step0 = w.u.first + (c.begin - w.u.start);
  w.r = range_of(w, w.s);
}

// x, y as bf16 pairs hi + lo
__device__ __forceinline__ void split(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 rest = ffma2(make_float2(bf_lo(hi), bf_hi(hi)), both(-1.f), x);
  lo = pack_bf16x2(rest.x, rest.y);
}
// the four pairs of centred codes of a word; the second and fourth times 16
__device__ __forceinline__ void centred(uint32_t w, float2 (&c)[4]) {
  const uint32_t y = w >> 8;
  const uint32_t h[4] = {hadd2(lop3_and_or(w, 0x000F000Fu, 0x64006400u), 0xE408E408u), hadd2(lop3_and_or(w, 0x00F000F0u, 0x64006400u), 0xE480E480u),
                         hadd2(lop3_and_or(y, 0x000F000Fu, 0x64006400u), 0xE408E408u), hadd2(lop3_and_or(y, 0x00F000F0u, 0x64006400u), 0xE480E480u)};
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
}

// Keys of 8 tokens (block b, half h) of a step: token row 16b + 8h + lane/4,
// channels 32g + 8i .. of every group, into the hi and lo boxes.
template <int D>
__device__ __forceinline__ void decode_keys(uint32_t raw, uint32_t keys, int b, int h, int64_t tok0, const Span& span) {
  constexpr int NG = D / 32, NBX = D / 64;
  const int lane = threadIdx.x & 31, i = lane & 3, t = 8 * h + (lane >> 2), row = 16 * b + t;
  const uint32_t blk = raw + b * kv_block_bytes(D), words = blk + (t * 4 + i) * (4 * NG), scales = blk + 16 * D + t * (2 * NG);
  const bool seen = tok0 + row >= span.first && tok0 + row <= span.last;
  // chunk 4*(g & 1) + i of 16 bytes, swizzled by the row: group g + 1 flips bit 2
  const uint32_t at = keys + row * 128 + ((i ^ (row & 7)) << 4);
#pragma unroll 1
  for (int g2 = 0; g2 < NG / 2; ++g2) {
    uint32_t w[2], sc[1], md[1];
    lds_words<2>(w, words + 8 * g2);
    lds_words<1>(sc, scales + 4 * g2);
    lds_words<1>(md, scales + D + 4 * g2);
    if (!seen) sc[0] = md[0] = 0;                               // it may hold anything
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float s = e ? bf_hi(sc[0]) : bf_lo(sc[0]), m = e ? bf_hi(md[0]) : bf_lo(md[0]), s16 = 0.0625f * s;
      float2 c[4];
      centred(w[e], c);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(ffma2(c[j], both(j & 1 ? s16 : s), both(m)), hi[j], lo[j]);
      const uint32_t to = (at ^ (e << 6)) + g2 * 8192;
      sts128(to, hi);
      sts128(to + NBX * 8192, lo);
    }
  }
}

// Values of a block's 64 channels 64*quad .. : words of channels d = 16mt +
// lane/4 and d + 8, tokens 2i, 2i+1, 2i+8, 2i+9, into the hi and lo rows d.
template <int D>
__device__ __forceinline__ void decode_values(Control& c, int j, uint32_t raw, uint32_t values, int b, int quad, int64_t tok0,
                                              const Span& span) {
  constexpr int NG = D / 32;
  const int lane = threadIdx.x & 31, i = lane & 3, q = lane >> 2;
  const uint32_t blk = raw + b * kv_block_bytes(D);
  const bool all = tok0 >= span.first && tok0 + kTok - 1 <= span.last;      // some row sees each token of the step
  // row d = 16 * tile + q (+ 8), chunks 2b and 2b + 1 of it, swizzled by q
  const uint32_t at = values + q * 128 + 4 * i, at0 = at + (((2 * b) ^ q) << 4), at1 = at + (((2 * b + 1) ^ q) << 4);
#pragma unroll 1
  for (int gg = 0; gg < 2; ++gg) {
    const int g = 2 * quad + gg;
    uint32_t w[2], md[2][1], bits[4];
    lds_words<2>(w, blk + 8 * D + (quad * 32 + lane) * 16 + 8 * gg);
    lds_words<1>(md[0], blk + 19 * D + g * 32 + 4 * i);
    lds_words<1>(md[1], blk + 19 * D + g * 32 + 4 * i + 16);
    const uint32_t scales = blk + 18 * D + (2 * i * NG + g) * 2;            // tokens 2i, 2i+1, 2i+8, 2i+9
#pragma unroll
    for (int k = 0; k < 4; ++k) bits[k] = lds_u16(scales + ((k & 1) + 8 * (k >> 1)) * (2 * NG));
    const bool odd = max(max(bits[0], bits[1]), max(bits[2], bits[3])) >= 0x7F80u;
    // 0 times a token that a row does not see has to be 0: those that no row
    // sees may hold anything, and a NaN reaches the rows that do see it through c.odd
    if (__any_sync(0xffffffffu, odd) || !all) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 16 * b + 2 * i + (k & 1) + 8 * (k >> 1);
        const int64_t tok = tok0 + t;
        const bool seen = tok >= span.first && tok <= span.last, bad = (bits[k] & 0x7F80u) == 0x7F80u;
        if (!seen || bad) {
          bits[k] = 0;
          md[k >> 1][0] &= k & 1 ? 0xFFFFu : 0xFFFF0000u;
        }
        if (seen && bad && q == 0) {
          c.odd[j & 1][g][t] = j + 1;
          c.odd_any[j & 1] = j + 1;
        }
      }
    }
    float2 s[2][2], m[2];                                       // and a sixteenth, for the codes that come as 16c
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      s[0][k] = make_float2(bf16_bits_to_f32(bits[2 * k]), bf16_bits_to_f32(bits[2 * k + 1]));
      s[1][k] = mul2(s[0][k], both(0.0625f));
      m[k] = make_float2(bf_lo(md[k][0]), bf_hi(md[k][0]));
    }
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      float2 x[4];
      centred(w[mm], x);
      const uint32_t tile = (2 * g + mm) * 2048;
#pragma unroll
      for (int j = 0; j < 4; ++j) {                             // j & 1: channel d + 8; j >> 1: tokens + 8
        uint32_t hi, lo;
        split(ffma2(x[j], s[j & 1][j >> 1], m[j >> 1]), hi, lo);
        const uint32_t to = (j >> 1 ? at1 : at0) + tile + (j & 1) * 1024;
        sts32(to, hi);
        sts32(to + D * 128, lo);
      }
    }
  }
}

template <int D, typename Out>
__global__ void __launch_bounds__(kThreads, 1) attention_block_kernel(const AttnArgs a) {
  using Y = Layout<D>;
  constexpr int NG = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Control& c = *reinterpret_cast<Control*>(smem + Y::kControlAt);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int k = tid; k < 2 * 4 * kTok; k += kThreads) c.odd[0][0][k] = 0;
  if (tid == 0) {
    for (int s = 0; s < kRawStages; ++s) mbar_init(&c.raw_full[s], 1), mbar_init(&c.raw_empty[s], kDecodeWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.k_full[s], kDecodeWarps), mbar_init(&c.k_empty[s], 1);
      mbar_init(&c.v_full[s], kDecodeWarps), mbar_init(&c.v_empty[s], 1);
      mbar_init(&c.q_ready[s], 4), mbar_init(&c.s_full[s], 1);
      mbar_init(&c.p_full[s], 4), mbar_init(&c.o_full[s], 1);
      c.odd_any[s] = 0;
    }
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) a.joined[blockIdx.x].parts = 0;
  const Plan pl = make_plan<kSB, kRows>(a, c.prefix, c.cost, nullptr);
  if (pl.total == 0 || blockIdx.x >= pl.ctas) return;
  if (tid < 2) (tid ? c.end : c.begin) = bound<kSB, kRows>(a, pl, blockIdx.x + tid);
  __syncthreads();
  if (c.begin >= c.end) return;
  const int steps = static_cast<int>(c.end - c.begin);
  Walk w;                                                        // the first piece, in code that all warps share
  w.end = 0;
  next_piece(a, pl, c, w, steps);
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c.tmem_base)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;

  int j = 0;                                                     // steps taken: buffers and phases go by it
  if (warp < kWarpSoft0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
  if (warp == kWarpLoad) {
    // ---- blocks of the cache into the raw ring; lane k < 4 copies a step's block k ----
    bool ok = true;
    for (; ok; next_piece(a, pl, c, w, steps)) {
      for (int n = w.r.lo; n < w.r.hi; ++n) {
        const int r = j % kRawStages;
        const uint8_t* src = nullptr;
        const int64_t blk = (w.step0 + n) * kSB + lane;
        if (lane < kSB && blk * kKvBlock < w.u.rq.L && (blk + 1) * kKvBlock > w.s.first) {
          src = kv_block_ptr(a.pool, a.kb, D, w.u.b, w.u.h, blk);
          if (src == nullptr) atomicOr(a.err, kErrIndex);
        }
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, src != nullptr)) * kv_block_bytes(D);
        if (!(ok = wait(c, &c.raw_empty[r], ((j / kRawStages) & 1) ^ 1, a.err))) break;
        if (lane == 0) mbar_arrive_expect_tx(&c.raw_full[r], bytes);
        __syncwarp();
        if (src != nullptr) bulk_g2s(smem + Y::kRawAt + r * Y::kRaw + lane * kv_block_bytes(D), src, kv_block_bytes(D), &c.raw_full[r]);
        ++j;
      }
      if (w.end >= steps) break;
    }
    for (int t = j > kRawStages ? j - kRawStages : 0; t < j; ++t)     // copies still under way land first
      mbar_wait_bounded(&c.raw_full[t % kRawStages], (t / kRawStages) & 1);
  } else if (warp == kWarpMma) {
    // ---- products; the whole warp runs the loop and its operands are broadcast, so
    // that they sit in uniform registers: issued from a single-lane branch the 28
    // products of a tile and step took 3200 cycles instead of 1800 ----
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t begun = 0, pending = 0, open = 0;                       // a bit per tile: phases of q_ready and s_full; p v to come; S formed in this piece
    uint32_t turn = 0;
    bool ok = true;
    for (; ok; next_piece(a, pl, c, w, steps)) {
      const Range r0 = range_of(w, span_of(a, w.u, 0, kTile)), r1 = range_of(w, span_of(a, w.u, kTile, kTile));
      uint32_t fresh = 0;                                            // nothing in O yet
      for (int n = w.r.lo; n <= w.r.hi && ok; ++n) {                 // and once more for the last p v
        const bool more = n < w.r.hi;
        bool keys = false;                                           // they are there
        const int b = __shfl_sync(0xffffffffu, j & 1, 0);
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          const uint32_t bit = 1u << t, cols = __shfl_sync(0xffffffffu, tm + t * Y::kCols, 0);
          if (pending & bit) {                                       // O (+)= p v of the step before, while the other tile's p are formed
            if (!(ok = wait(c, &c.p_full[t], (turn >> t & 1) ^ 1, a.err))) break;      // whose warps have waited for this step's v_full
            tc_fence_after();
            const uint64_t v = sw128_desc(base + Y::kValuesAt + (b ^ 1) * Y::kValues);
            const uint32_t p = cols + Y::kS, o = cols + Y::kO;
            mma64<idesc(D), 8, 32, 40>(o, p, v, !(fresh & bit));     // p_hi v_hi
            mma64<idesc(D), 8, 32, 40>(o, p + 16, v, 1);             // p_lo v_hi
            mma64<idesc(D), 8, 32, 40>(o, p, v + D * 128 / 16, 1);   // p_hi v_lo
            pending ^= bit, fresh &= ~bit;
          }
          if (t == 1 && n > w.r.lo) commit(&c.v_empty[b ^ 1]);       // the step before is done with: its values' place
          if (!more) {
            if (open & bit) commit(&c.o_full[t]);
          } else if (n >= (t ? r1.lo : r0.lo) && n < (t ? r1.hi : r0.hi)) {
            if (!(open & bit)) {
              if (!(ok = wait(c, &c.q_ready[t], begun >> t & 1, a.err))) break;
              open |= bit, fresh |= bit, begun ^= bit;
            }
            if (!keys && !(ok = keys = wait(c, &c.k_full[b], (j >> 1) & 1, a.err))) break;
            tc_fence_after();
            const uint64_t k = sw128_desc(base + b * Y::kKeys);
#pragma unroll
            for (int x = 0; x < 2 * Y::NBX; ++x)                     // boxes of 64 channels, those of hi, then of lo
              mma64<idesc(kTok), 8, 16, 24>(cols + Y::kS, cols + Y::kQ + 32 * (x % Y::NBX), k + x * 512, x > 0);
            commit(&c.s_full[t]);
            pending ^= bit, turn ^= bit;
          }
        }
        if (!ok) break;
        if (more) {
          commit(&c.k_empty[b]);
          ++j;
        }
      }
      open = 0;
      if (w.end >= steps) break;
    }
    commit(&c.drain);                                                // every product issued so far has completed
    mbar_wait_bounded(&c.drain, 0, 100000000ull);
  } else if (warp >= kWarpDecode0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
    // ---- codes to bf16 pairs: warp d decodes keys of block d/2, half d%2, and values of its channels 64*(d%2) .. ----
    const int d = warp - kWarpDecode0, blk = d >> 1, half = d & 1;
    bool ok = true;
    for (; ok; next_piece(a, pl, c, w, steps)) {
      for (int n = w.r.lo; n < w.r.hi; ++n) {
        const int b = j & 1, r = j % kRawStages;
        const int64_t t0 = (w.step0 + n) * kTok;
        const uint32_t raw = base + Y::kRawAt + r * Y::kRaw, free_phase = ((j >> 1) & 1) ^ 1;
        if (!(ok = wait(c, &c.raw_full[r], (j / kRawStages) & 1, a.err) && wait(c, &c.k_empty[b], free_phase, a.err))) break;
        decode_keys<D>(raw, base + b * Y::kKeys, blk, half, t0, w.s);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive(&c.k_full[b]);
        if (!(ok = wait(c, &c.v_empty[b], free_phase, a.err))) break;
        if (half < D / 64) decode_values<D>(c, j, raw, base + Y::kValuesAt + b * Y::kValues, blk, half, t0, w.s);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          arrive(&c.v_full[b]);
          arrive(&c.raw_empty[r]);
        }
        ++j;
      }
      if (w.end >= steps) break;
    }
  } else if (warp >= kWarpSoft0) {
    // ---- softmax, four warps a tile: a thread is a row ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int t = (warp - kWarpSoft0) >> 2, row = kTile * t + 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + t * Y::kCols + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    int turn = 0;                                                    // steps of the tile
    int piece = 0;
    const float none = -__int_as_float(0x7f800000), c2 = a.scale_log2;
    bool ok = true;
    for (; ok; next_piece(a, pl, c, w, steps)) {
      const int64_t x0 = c.begin + w.at, row0 = w.u.rg * kRows, left = w.u.rq.T * a.group - row0;
      const bool have = row < w.s.rows;                              // those that have none take the last, and keep nothing of it
      const int64_t r = row0 + (row < left ? row : left - 1), tq = quot(r, a.group), head = w.u.h * a.group + (r - tq * a.group);
      const int64_t pos = w.u.rq.L - w.u.rq.T + tq;
      const int64_t hi = pos < w.u.rq.L ? pos : w.u.rq.L - 1;                               // the row sees lo < position <= hi
      const int64_t lo = a.window > 0 && pos - a.window > -1 ? pos - a.window : -1;
      // the positions that all rows of the warp see; later rows see from and to later ones
      const int64_t all_lo = __shfl_sync(0xffffffffu, lo, 31), all_hi = __shfl_sync(0xffffffffu, hi, 0);
      const Range own = range_of(w, span_of(a, w.u, kTile * t, kTile));
      // the query row into TMEM (bf16 pairs, a column each); the piece before has no products left that read it
      const uint4* q = reinterpret_cast<const uint4*>(a.q + (w.u.rq.q0 + tq) * a.q_stride + head * D);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t v[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 x = __ldg(q + 8 * h + k);
          v[4 * k] = x.x, v[4 * k + 1] = x.y, v[4 * k + 2] = x.z, v[4 * k + 3] = x.w;
        }
        tmem_store(lanes + Y::kQ + 32 * h, v);
      }
      tmem_wait_store();
      tc_fence_before();
      __syncwarp();
      bool begun = false;
      float ref = kRefNone, l = 0.f;
      uint32_t odd = 0;                                             // groups in which the row has seen a NaN
      j += own.lo - w.r.lo;
      for (int n = own.lo; n < own.hi; ++n, ++j) {
        const int b = j & 1;
        if (!begun && lane == 0) arrive(&c.q_ready[t]);
        const int64_t t0 = (w.step0 + n) * kTok;
        const bool part = t0 <= all_lo || t0 + kTok - 1 > all_hi;
        int from = 0, to = kTok;                                    // sees from <= k < to
        if (part) {
          from = static_cast<int>(lo - t0 + 1 > 0 ? (lo - t0 + 1 < kTok ? lo - t0 + 1 : kTok) : 0);
          to = static_cast<int>(hi - t0 + 1 < kTok ? (hi - t0 + 1 > 0 ? hi - t0 + 1 : 0) : kTok);
        }
        // S first, then the values, of which the product (issued on p_full) and `odd` need
        // the latter.  The order matters: a tile goes past steps that its rows do not see
        // without a wait, and parity tells v_full's phases apart only one step of a buffer
        // away.  S of this step means that all decoding warps have posted the values of
        // the steps before, so that the phase awaited is the current one or the last.
        if (!(ok = wait(c, &c.s_full[t], turn++ & 1, a.err) && wait(c, &c.v_full[b], (j >> 1) & 1, a.err))) break;
        if (c.odd_any[b] == j + 1) {
          for (int g = 0; g < NG; ++g)
            for (int k = from; k < to; ++k)
              if (c.odd[b][g][k] == j + 1) odd |= 1u << g;
        }
        __syncwarp();
        tc_fence_after();
        // the row's 64 logits stay in registers between maximum and weights: read again
        // for the second pass they cost 64.5 us instead of 62
        uint32_t x[2][32];
        tmem_load(lanes + Y::kS, x[0]);
        tmem_load(lanes + Y::kS + 32, x[1]);
        tmem_wait_load(x[0]);
        tmem_wait_load(x[1]);
        float top = none, mul = c2;
        if (part || c2 <= 0.f) {
          mul = 1.f;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float y = k + 32 * h < from || k + 32 * h >= to ? none : __uint_as_float(x[h][k]) * c2;
              x[h][k] = __float_as_uint(y);
              top = fmaxf(top, y);
            }
        } else {
          float m[4] = {none, none, none, none};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              m[k / 2 & 3] = fmaxf(m[k / 2 & 3], fmaxf(__uint_as_float(x[h][k]), __uint_as_float(x[h][k + 1])));
          top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c2;
        }
        const bool move = top > ref + 8.f;
        if (__any_sync(0xffffffffu, move)) {
          const float now = move ? top : ref, f = ex2(ref - now);
          ref = now;
          l *= f;
          if (begun) {                                               // O: the products before S are in it
#pragma unroll 1
            for (int h = 0; h < D / 16; ++h) {
              uint32_t o[16];
              tmem_load16(lanes + Y::kO + 16 * h, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_store16(lanes + Y::kO + 16 * h, o);
            }
            tmem_wait_store();
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p_hi[16], p_lo[16];
          float2 sum = both(0.f);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 y = ex2(ffma2(make_float2(__uint_as_float(x[h][2 * k]), __uint_as_float(x[h][2 * k + 1])), both(mul), both(-ref)));
            sum = fadd2(sum, y);
            split(y, p_hi[k], p_lo[k]);
          }
          l += sum.x + sum.y;
          tmem_store16(lanes + Y::kS + 32 * h, p_hi);
          tmem_store16(lanes + Y::kS + 32 * h + 16, p_lo);
        }
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(&c.p_full[t]);
        begun = true;
      }
      if (!ok) break;
      j += w.r.hi - own.hi;
      if (begun && !(ok = wait(c, &c.o_full[t], piece++ & 1, a.err))) break;
      tc_fence_after();
      // O to the output, or as a part to the workspace
      const bool whole = x0 == w.u.start && w.end == w.u.start + w.u.n - c.begin, first = w.u.start >= c.begin;
      float* part = a.partial + static_cast<int64_t>(2 * blockIdx.x + (first ? 1 : 0)) * kRows * (D + 2);
      const int64_t at = (w.u.rq.q0 + tq) * a.heads + head;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int h = 0; h < D / 32; ++h) {
        uint32_t o[32];
        if (begun) {
          tmem_load(lanes + Y::kO + 32 * h, o);
          tmem_wait_load(o);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (!begun || l == 0.f) o[k] = 0;
        if (odd >> h & 1)
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0x7fc00000u;
        if (have && whole) {
          if constexpr (sizeof(Out) == 4) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D + 32 * h + k) =
                  make_float4(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv, __uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + 32 * h + k) =
                  make_uint4(pack_bf16x2(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv),
                             pack_bf16x2(__uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv),
                             pack_bf16x2(__uint_as_float(o[k + 4]) * inv, __uint_as_float(o[k + 5]) * inv),
                             pack_bf16x2(__uint_as_float(o[k + 6]) * inv, __uint_as_float(o[k + 7]) * inv));
          }
        } else if (have) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)                             // [D / 4][row][4]: a warp's rows side by side
            *reinterpret_cast<uint4*>(part + ((8 * h + k / 4) * kRows + row) * 4) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      tc_fence_before();
      if (have && whole && a.lse != nullptr) a.lse[at] = log_total(ref, l);
      if (have && !whole) *(reinterpret_cast<float2*>(part + kRows * D) + row) = make_float2(ref, l);
      if (!whole && first && row == 0) {
        // this CTA has the unit's first part: the others are those of the next CTAs up to the unit's end
        const int c1 = share_of(pl, w.u.cost + kUnitCost + w.u.n - cut_steps<kRows>);
        a.joined[blockIdx.x] = {w.u.rq.q0, w.u.rg * kRows, w.u.h, w.s.rows, c1 - static_cast<int>(blockIdx.x) + 1, 0};
      }
      if (w.end >= steps) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// The parts of units cut between CTAs: a thread per row and four channels, lanes
// along the rows, as the parts lie.
constexpr int kJoinWarps = 8;

template <int D, typename Out>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const AttnArgs a) {
  constexpr int kBatch = 10;
  constexpr int64_t kPitch = kRows * (D + 2);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Joined u = a.joined[blockIdx.x];
  const int slot = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), r = slot % (kRows / 32) * 32 + (threadIdx.x & 31), c4 = slot / (kRows / 32);
  if (u.parts == 0 || r >= u.rows) return;
  auto part = [&](int c) { return a.partial + (2 * (blockIdx.x + c) + (c == 0 ? 1 : 0)) * kPitch; };
  float m = kRefNone, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c = 0; c < u.parts; c += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* from = part(c + k < u.parts ? c + k : c);
      ml[k] = __ldcg(reinterpret_cast<const float2*>(from + kRows * D) + r);
      v[k] = __ldcg(reinterpret_cast<const float4*>(from) + c4 * kRows + r);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);           // a part taken twice changes no maximum
    const float f0 = ex2(m - top);
    m = top, l *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (c + k < u.parts) {
        const float f = ex2(ml[k].x - m);
        l = fmaf(f, ml[k].y, l);
        o.x = fmaf(f, v[k].x, o.x), o.y = fmaf(f, v[k].y, o.y), o.z = fmaf(f, v[k].z, o.z), o.w = fmaf(f, v[k].w, o.w);
      }
  }
  const int64_t at = out_row(a, u.q0, u.h, u.row0 + r);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (sizeof(Out) == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D + 4 * c4) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + 4 * c4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (c4 == 0 && a.lse != nullptr) a.lse[at] = log_total(m, l);
}

template <int D, typename Out>
cudaError_t launch_block_variant(const AttnArgs& a, int grid, cudaStream_t s) {
  static_assert(kSmemBytes<D> <= 232448, "shared memory per CTA");
  const void* f = reinterpret_cast<const void*>(attention_block_kernel<D, Out>);
  cudaError_t e = set_max_dynamic_smem(f);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes<D>;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attention_block_kernel<D, Out>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), kRows / 32 * (D / 4) / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<D, Out>, a);
}

}  // namespace

uint64_t attention_block_bytes(int D) { return D > 128 ? 0 : static_cast<uint64_t>(kKvMaxCtas) * kRows * (D + 2) * 4; }

cudaError_t launch_attention_block(int D, const AttnArgs& a, int out_f32, const DeviceInfo& info, cudaStream_t s) {
  const int grid = info.sms < kKvMaxCtas / 2 ? info.sms : kKvMaxCtas / 2;      // two parts each
  switch (D) {
    case 64: return out_f32 ? launch_block_variant<64, float>(a, grid, s) : launch_block_variant<64, uint16_t>(a, grid, s);
    case 128: return out_f32 ? launch_block_variant<128, float>(a, grid, s) : launch_block_variant<128, uint16_t>(a, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace q4nx
