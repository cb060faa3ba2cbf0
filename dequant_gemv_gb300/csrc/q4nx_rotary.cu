// q4nx_rotary.cu -- new queries and keys turned by their positions, the keys and the
// values on into the 4-bit cache (layout and value formula: q4nx_kv.cuh).
//
// A pair of channels (a, b) of a head, at a token with cosine c and sine s of the pair:
//   a' = a c - b s,  b' = b c + a s,
// every product, difference and sum one IEEE binary32 operation, so that every machine
// takes the same codes.  Keys go from there into codes as in q4nx_kv.cu, without a rounding to
// bf16 between, but that a group's range is multiplied by 1/15 instead of divided (scale_of); queries leave as bf16.  Cosines and sines come from the caller's
// table: they are made once in 64 bits (positions times frequencies lose their angle
// in 32), and a token's 8 bytes a pair are shared by all of its heads.
//
// Two kernels, as without the rotation: few tokens per request take a warp per (token, kv
// head) and per (token, query head); prompts a CTA per 16-token block of the cache and
// some of the heads, with the block's cosines and sines in shared memory for its keys, and in
// a thread's registers, which turns the same channels of many heads, for its queries.
//
// Bound.  3 prompts of up to 1501 tokens, 32 query and 8 kv heads of 128 (2854 tokens): 19 to 20.5 us, keys
// and values alone 12 to 19 from run to run.  64 MB with the cosines: 3.1 to 3.4 TB/s, half of a copy's rate.  A key or value costs about 44
// instructions of a lane (turn, extremes, code with its exact ties), the queries' 47 MB come on top: the two
// parts run beside one another only where one ends, and their CTAs alternating in the grid took 21.6 us
// (query rows no longer in order), five CTAs an SM no less.  A CTA's 16 query heads: 18.9; 8: 19.5; 4: 22.2
// (the look-up again for each).  Two numbers an instruction (packed binary32), ties by one test for both: 36, with the
// rare way's code in the loop.  One token for each of 48 requests: 3.9 us, a launch and look-ups in series.
#include "q4nx_kernels.h"
#include "q4nx_kv_store.cuh"

namespace q4nx {

namespace {

constexpr int kWarps = 8;
constexpr int64_t kFullItems = 16384;  // (token, head) pairs, queries and keys, from which on there are blocks enough

struct TurnArgs {
  KvPool pool;
  KvBatch kb;
  RotaryCall c;
};

// own * c -/+ other * s: the first or the second channel of a pair
__device__ __forceinline__ float turned(float own, float other, float2 cs, bool second) {
  const float x = __fmul_rn(own, cs.x), y = __fmul_rn(other, cs.y);
  return second ? __fadd_rn(x, y) : __fsub_rn(x, y);
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A head of the token at position pos, lane l with channels VPL*l .., as numbers, turned.
template <int D>
__device__ __forceinline__ void turn_token(const RotaryCall& c, int64_t pos, const uint32_t (&raw)[D / 64], float (&x)[D / 32]) {
  constexpr int VPL = D / 32;
  const int lane = threadIdx.x & 31, d0 = lane * VPL;
  const bool in = d0 < 2 * c.half;
#pragma unroll
  for (int j = 0; j < VPL / 2; ++j) x[2 * j] = lo16(raw[j]), x[2 * j + 1] = hi16(raw[j]);
  const float2* row = c.table + pos * c.half;
  if (c.interleaved) {
    if (in)
#pragma unroll
      for (int j = 0; j < VPL / 2; ++j) {
        const float2 cs = __ldg(row + d0 / 2 + j);
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = turned(a, b, cs, false);
        x[2 * j + 1] = turned(b, a, cs, true);
      }
    return;
  }
  const bool second = d0 >= c.half;
  const int step = c.half / VPL, from = in ? (second ? lane - step : lane + step) : lane;
  float2 cs[VPL];
#pragma unroll
  for (int j = 0; j < VPL; j += 2) {
    const float4 two = in ? __ldg(reinterpret_cast<const float4*>(row + (second ? d0 - c.half : d0) + j)) : make_float4(1.f, 0.f, 1.f, 0.f);
    cs[j] = make_float2(two.x, two.y), cs[j + 1] = make_float2(two.z, two.w);
  }
#pragma unroll
  for (int j = 0; j < VPL / 2; ++j) {
    const uint32_t other = __shfl_sync(0xffffffffu, raw[j], from);
    if (in) {
      x[2 * j] = turned(x[2 * j], lo16(other), cs[2 * j], second);
      x[2 * j + 1] = turned(x[2 * j + 1], hi16(other), cs[2 * j + 1], second);
    }
  }
}

// One warp per (token, kv head) and per (token, query head).
template <int D>
__global__ void __launch_bounds__(kWarps * 32) turn_tokens_kernel(const TurnArgs a) {
  constexpr int VPL = D / 32;
  __shared__ __align__(16) uint8_t codes[kWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RotaryCall& c = a.c;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int per = a.pool.kv_heads + c.heads;
  const int64_t tok = item / per;
  const int unit = static_cast<int>(item - tok * per), h = unit - a.pool.kv_heads;       // h below 0: a kv head
  if (tok >= a.kb.tokens) {
    if (tok == a.kb.tokens && unit == 0) kv_report(a.kb, a.pool.page_blocks, c.err);
    return;
  }
  uint32_t raw[2][VPL / 2];                                     // the values, ahead of the look-ups
  {
    const uint16_t* k = h < 0 ? c.k + tok * c.kv_stride + static_cast<int64_t>(unit) * D : c.q + tok * c.q_stride + static_cast<int64_t>(h) * D;
#pragma unroll
    for (int j = 0; j < VPL / 2; ++j) raw[0][j] = reinterpret_cast<const uint32_t*>(k + lane * VPL)[j];
    if (h < 0)
#pragma unroll
      for (int j = 0; j < VPL / 2; ++j)
        raw[1][j] = __ldg(reinterpret_cast<const uint32_t*>(c.v + tok * c.kv_stride + static_cast<int64_t>(unit) * D + lane * VPL) + j);
  }
  int b;
  const KvRequest rq = kv_locate(a.kb, a.pool.page_blocks, tok, b);
  if (b < 0) return;                                            // a token of no request
  const int64_t pos = rq.L - rq.T + (tok - rq.q0);
  if (!rq.ok || pos >= c.positions) {
    if (lane == 0) atomicOr(c.err, kErrIndex);
    return;
  }
  if (pos < 0) return;
  float x[VPL];
  if (h >= 0) {
    turn_token<D>(c, pos, raw[0], x);
    uint32_t* to = reinterpret_cast<uint32_t*>(c.q_out + tok * c.q_out_stride + static_cast<int64_t>(h) * D + lane * VPL);
    if constexpr (VPL == 8) {
      *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else if constexpr (VPL == 4) {
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    } else {
      *to = pack_bf16x2(x[0], x[1]);
    }
    return;
  }
  uint8_t* blk = kv_block_ptr(a.pool, a.kb, D, b, unit, pos / kKvBlock);
  if (blk == nullptr) {
    if (lane == 0) atomicOr(c.err, kErrIndex);
    return;
  }
  const int t = static_cast<int>(pos % kKvBlock);
  turn_token<D>(c, pos, raw[0], x);
  keep_token<D>(blk, t, 0, true, x, codes[warp]);
#pragma unroll
  for (int j = 0; j < VPL / 2; ++j) x[2 * j] = lo16(raw[1][j]), x[2 * j + 1] = hi16(raw[1][j]);
  keep_token<D>(blk, t, 1, false, x, codes[warp]);
}

// A CTA per 16-token block that the call writes and part of the heads: kv heads first
// (kKvHeads of them a CTA), then query heads (kQHeads).
template <int D>
constexpr int kKvHeads = D == 256 ? 2 : D == 128 ? 4 : 8;
constexpr int kQHeads = 16;

// Whether a lane that holds a group of 32 channels finds their partners in it or in its neighbour lane's.
__host__ __device__ __forceinline__ bool by_groups(int half, bool interleaved) { return interleaved || half % 32 == 0 || half == 16; }

template <int D>
__global__ void __launch_bounds__(kWarps * 32) turn_blocks_kernel(const TurnArgs a) {
  constexpr int NG = D / 32, kRow = D / 2 + 2;                  // a token's pairs; two more, so that tokens lie on different banks
  __shared__ __align__(16) float2 table[kKvBlock][kRow];
  __shared__ __align__(16) uint8_t image[kWarps][512];          // value codes of two groups of a block
  __shared__ struct {
    int64_t q0, T, L, blk;
    int b;
  } at;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RotaryCall& c = a.c;
  if (warp == 0) {
    int64_t left = blockIdx.x;
    if (left == most_blocks(a.kb)) {
      if (blockIdx.y == 0) kv_report(a.kb, a.pool.page_blocks, c.err);
      left = INT64_MAX;
    }
    int b = -1;
    KvRequest rq = {};
    if (left != INT64_MAX) rq = locate_block(a.kb, a.pool.page_blocks, left, b);
    if (lane == 0) at.q0 = rq.q0, at.T = rq.T, at.L = rq.L, at.blk = (rq.L > rq.T ? rq.L - rq.T : 0) / kKvBlock + left, at.b = b;
  }
  __syncthreads();
  if (at.b < 0) return;
  const KvRequest rq = {at.q0, at.T, at.L, true};
  const int64_t blk_at = at.blk, from = rq.L > rq.T ? rq.L - rq.T : 0, p0 = blk_at * kKvBlock;
  const int64_t end = rq.L < c.positions ? rq.L : c.positions;  // positions from `from` to here have a place in cache and table
  const int first = static_cast<int>(from > p0 ? from - p0 : 0), last = static_cast<int>(end - p0 < kKvBlock ? (end > p0 ? end - p0 : 0) : kKvBlock);
  if (tid == 0 && p0 + kKvBlock > c.positions && rq.L > c.positions) atomicOr(c.err, kErrIndex);
  const int64_t tok0 = rq.q0 + p0 - (rq.L - rq.T);              // the token of position p0, if it is the call's
  const int ykv = (a.pool.kv_heads + kKvHeads<D> - 1) / kKvHeads<D>;
  if (blockIdx.y >= ykv) {
    // ---- queries: a thread turns 8 pairs (or moves 8 channels) of one token in every second, fourth .. head ----
    const int half8 = c.interleaved ? D / 8 : c.half / 8, per = c.interleaved ? D / 8 : half8 + (D - 2 * c.half) / 8;
    const int h0 = (blockIdx.y - ykv) * kQHeads, heads = c.heads - h0 < kQHeads ? c.heads - h0 : kQHeads;
    const int ways = kWarps * 32 / (kKvBlock * per) > 0 ? kWarps * 32 / (kKvBlock * per) : 1;   // heads at a time
#pragma unroll 1
    for (int i = tid; i < kKvBlock * per * ways; i += kWarps * 32) {
      const int chunk = i % per, t = i / per % kKvBlock, way = i / (per * kKvBlock);
      if (t < first || t >= last) continue;
      const int64_t tok = tok0 + t;
      const bool plain = c.interleaved ? 8 * chunk >= 2 * c.half : chunk >= half8;
      const int d = c.interleaved || !plain ? 8 * chunk : 2 * c.half + 8 * (chunk - half8);
      const uint16_t* q = c.q + tok * c.q_stride + static_cast<int64_t>(h0) * D + d;
      uint16_t* o = c.q_out + tok * c.q_out_stride + static_cast<int64_t>(h0) * D + d;
      if (plain) {
#pragma unroll 4
        for (int h = way; h < heads; h += ways) *reinterpret_cast<uint4*>(o + h * D) = *reinterpret_cast<const uint4*>(q + h * D);
        continue;
      }
      float2 cs[8];
      const float2* row = c.table + (p0 + t) * c.half + (c.interleaved ? 4 * chunk : 8 * chunk);
      if (c.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const float4 two = __ldg(reinterpret_cast<const float4*>(row + j));
          cs[j] = make_float2(two.x, two.y), cs[j + 1] = make_float2(two.z, two.w);
        }
#pragma unroll 4
        for (int h = way; h < heads; h += ways) {
          const uint4 w = *reinterpret_cast<const uint4*>(q + h * D);
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) r[j] = pack_bf16x2(turned(lo16(v[j]), hi16(v[j]), cs[j], false), turned(hi16(v[j]), lo16(v[j]), cs[j], true));
          *reinterpret_cast<uint4*>(o + h * D) = make_uint4(r[0], r[1], r[2], r[3]);
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float4 two = __ldg(reinterpret_cast<const float4*>(row + j));
        cs[j] = make_float2(two.x, two.y), cs[j + 1] = make_float2(two.z, two.w);
      }
#pragma unroll 4
      for (int h = way; h < heads; h += ways) {
        const uint4 wa = *reinterpret_cast<const uint4*>(q + h * D), wb = *reinterpret_cast<const uint4*>(q + h * D + c.half);
        const uint32_t va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
        uint32_t ra[4], rb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ra[j] = pack_bf16x2(turned(lo16(va[j]), lo16(vb[j]), cs[2 * j], false), turned(hi16(va[j]), hi16(vb[j]), cs[2 * j + 1], false));
          rb[j] = pack_bf16x2(turned(lo16(vb[j]), lo16(va[j]), cs[2 * j], true), turned(hi16(vb[j]), hi16(va[j]), cs[2 * j + 1], true));
        }
        *reinterpret_cast<uint4*>(o + h * D) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
        *reinterpret_cast<uint4*>(o + h * D + c.half) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
      }
    }
    return;
  }
  // ---- keys and values ----
  for (int i = tid; i < kKvBlock * c.half / 2; i += kWarps * 32) {
    const int t = i / (c.half / 2), j = 2 * (i - t * (c.half / 2));
    if (t >= first && t < last)
      *reinterpret_cast<float4*>(&table[t][j]) = __ldg(reinterpret_cast<const float4*>(c.table + (p0 + t) * c.half + j));
  }
  __syncthreads();
  const int h0 = blockIdx.y * kKvHeads<D>, heads = a.pool.kv_heads - h0 < kKvHeads<D> ? a.pool.kv_heads - h0 : kKvHeads<D>;
  const int t = lane >> 1, e = lane & 1, HG = c.interleaved ? 0 : c.half / 32;
  const bool mine = t >= first && t < last;
#pragma unroll 1
  for (int item = warp; item < heads * NG; item += kWarps) {
    const int h = h0 + item / NG, which = item % NG / (NG / 2), pair = item % (NG / 2);
    uint8_t* blk = kv_block_ptr(a.pool, a.kb, D, at.b, h, blk_at);
    if (blk == nullptr) {
      if (lane == 0) atomicOr(c.err, kErrIndex);
      return;
    }
    // keys: the groups of a pair are partners where whole groups are
    const bool across = which == 0 && pair < HG;
    const int g = across ? pair + e * HG : 2 * pair + e;
    const uint16_t* src = (which ? c.v : c.k) + (mine ? tok0 + t : rq.q0) * c.kv_stride + static_cast<int64_t>(h) * D + 32 * g;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = mine ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0, 0, 0, 0);
      w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
    }
    float x[32];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[2 * j] = lo16(w[j]), x[2 * j + 1] = hi16(w[j]);
    if (across) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 cs = *reinterpret_cast<const float4*>(&table[t][32 * pair + 2 * j]);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, w[j], 1);
        x[2 * j] = turned(x[2 * j], lo16(other), make_float2(cs.x, cs.y), e);
        x[2 * j + 1] = turned(x[2 * j + 1], hi16(other), make_float2(cs.z, cs.w), e);
      }
    } else if (which == 0 && c.interleaved) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (16 * g + j < c.half) {
          const float2 cs = table[t][16 * g + j];
          x[2 * j] = turned(lo16(w[j]), hi16(w[j]), cs, false);
          x[2 * j + 1] = turned(hi16(w[j]), lo16(w[j]), cs, true);
        }
    } else if (which == 0 && c.half == 16 && g == 0) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 cs = table[t][j];
        const float p = x[j], r = x[j + 16];
        x[j] = turned(p, r, cs, false);
        x[j + 16] = turned(r, p, cs, true);
      }
    }
    float lo = x[0], hi = x[0];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
      bad |= !(fabsf(x[j]) < __int_as_float(0x7f800000));
    }
    keep_group<D>(blk, first == 0 && last == kKvBlock, mine, t, g, which, which == 0, lo, hi, bad, [&](int j) { return x[j]; }, image[warp]);
    __syncwarp();                                               // the image is read out
  }
}

template <int D>
cudaError_t launch_turn(const TurnArgs& a, cudaStream_t s) {
  const int kv = a.pool.kv_heads;
  // By blocks from 8 tokens per request on average on, where there are enough of them.  32 query and 8 kv heads of
  // 128, requests x tokens, by tokens and by blocks: 1 x 256 6.5 and 8.7 us, 1 x 512 9.9 and 8.7 to 9.8,
  // 16 x 32 9.7 and 9.5, 1 x 1024 16.0 and 9.5, 1 x 4096 55 and 26; 48 x 5 6.4 and 16, 32 x 24 12.6 and
  // 10.8, 64 x 16 16 and 12, 256 x 8 35 and 31; keys alone: 1 x 1024 7.8 and 15, 1 x 2048 12.5 and 10 to 15; 16
  // and 4 of 256: 1 x 512 8.4 and 15, 1 x 1024 13.1 and 10.5 to 15, 1 x 2048 22 and 12 to 16; 32 and 8 of 64: 1 x 512 8.8
  // and 8.2.  (By blocks a call has two times, 5 us apart, of which a process shows one or the other.)  Rotations whose
  // pairs by_groups does not find are by tokens at any size: 48 of 128 channels turned, 1 x 4096 55 us.
  if (by_groups(a.c.half, a.c.interleaved) && a.kb.tokens >= static_cast<int64_t>(8) * a.kb.batch && a.kb.tokens * (kv + a.c.heads) >= kFullItems) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(most_blocks(a.kb) + 1),       // and one that reports what is out of range
                       static_cast<unsigned>((kv + kKvHeads<D> - 1) / kKvHeads<D> + (a.c.heads + kQHeads - 1) / kQHeads));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, turn_blocks_kernel<D>, a);
  }
  const int64_t grid = a.kb.tokens * (kv + a.c.heads) / kWarps + 1;         // and a warp that reports
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch(turn_tokens_kernel<D>, static_cast<unsigned>(grid), kWarps * 32, 0, s, a);
}

}  // namespace

cudaError_t launch_kv_append_rotary(int D, const KvPool& p, const KvBatch& kb, const RotaryCall& c, cudaStream_t s) {
  const TurnArgs a = {p, kb, c};
  switch (D) {
    case 64: return launch_turn<64>(a, s);
    case 128: return launch_turn<128>(a, s);
    case 256: return launch_turn<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace q4nx
