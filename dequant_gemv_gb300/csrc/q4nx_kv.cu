// q4nx_kv.cu -- new keys and values into the 4-bit cache, and cached ones back
// out of it (layout and value formula: q4nx_kv.cuh).
//
// Quantisation of 32 values x of one token and head, each step one IEEE
// binary32 operation, so that every machine takes the same codes:
//   lo, hi = min, max;  scale = bf16((hi - lo) / 15);  mid = bf16(lo + 8*scale)
//   code = clamp(rint((x - mid) / scale), -8, 7) + 8   (ties to even; 8 where scale is 0)
// A group that holds a NaN or an infinity, or whose range overflows, keeps NaN
// as its scale and mid: all of it reads as NaN.
//
// Two append kernels: few tokens per request take a warp per (token, kv head),
// all lanes on one token's channels; prompts take a warp per (16-token block,
// kv head, keys or values, 64 channels), which owns them during the launch and writes whole
// sectors (a token's value codes are one byte in each of 64 words: 3351 tokens of
// 8 heads by the first kernel 16.1 us, by the second 10.7).  Floor: bytes (2 in, 0.625
// out per value, 2.7 us of these); what keeps it from them are latencies: the request's look-up
// before the loads, a lane's 64 bytes apart from the next lane's, 2-byte stores of scales.
#include "q4nx_kernels.h"
#include "q4nx_kv_store.cuh"

namespace q4nx {

namespace {

constexpr int kKvWarps = 8;      // warps per CTA of the append and read kernels
constexpr int64_t kFullItems = 6144;   // (token, head) pairs from which on larger items pay: below, too few warps have work

// One warp per (token, kv head).  Lane l holds channels VPL*l .. of the head.
template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_append_kernel(KvPool pool, KvBatch kb, const uint16_t* __restrict__ k,
                                                                 const uint16_t* __restrict__ v, int64_t stride,
                                                                 uint32_t* err) {
  constexpr int VPL = D / 32;                                   // values per lane
  __shared__ __align__(16) uint8_t codes[kKvWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kKvWarps + warp;
  const int64_t tok = item / pool.kv_heads;
  const int h = static_cast<int>(item - tok * pool.kv_heads);
  if (tok >= kb.tokens) {
    if (tok == kb.tokens && h == 0) kv_report(kb, pool.page_blocks, err);
    return;
  }
  uint32_t raw[2][VPL / 2];                                     // the values, ahead of the look-ups
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int j = 0; j < VPL / 2; ++j)
      raw[which][j] = __ldg(reinterpret_cast<const uint32_t*>((which ? v : k) + tok * stride + static_cast<int64_t>(h) * D + lane * VPL) + j);
  int b;
  const KvRequest rq = kv_locate(kb, pool.page_blocks, tok, b);
  if (b < 0) return;                                            // a token of no request
  const int64_t pos = rq.L - rq.T + (tok - rq.q0);
  uint8_t* blk = nullptr;
  if (rq.ok && pos >= 0) blk = kv_block_ptr(pool, kb, D, b, h, pos / kKvBlock);
  if (blk == nullptr) {
    if ((!rq.ok || pos >= 0) && lane == 0) atomicOr(err, kErrIndex);
    return;
  }
  const int t = static_cast<int>(pos % kKvBlock);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float x[VPL];
#pragma unroll
    for (int j = 0; j < VPL; j += 2) {
      const uint32_t w = raw[which][j / 2];
      x[j] = bf16_bits_to_f32(w & 0xFFFF);
      x[j + 1] = bf16_bits_to_f32(w >> 16);
    }
    keep_token<D>(blk, t, which, false, x, codes[warp]);
  }
}

// One warp per (16-token block that the call writes, kv head, keys or values,
// pair of groups): lane 2t + e holds one group of token t, so that no lane
// needs another's extremes.  Keys' words are stored as they come; values' bytes, 512
// in a row, are gathered in shared memory first.
template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_append_blocks_kernel(KvPool pool, KvBatch kb, const uint16_t* __restrict__ k,
                                                                        const uint16_t* __restrict__ v, int64_t stride,
                                                                        uint32_t* err) {
  constexpr int NG = D / 32;
  __shared__ __align__(16) uint8_t image[kKvWarps][512];        // value codes of the block's two groups
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kKvWarps + warp;
  const int which = static_cast<int>(item % NG) / (NG / 2), pair = static_cast<int>(item % (NG / 2));
  int64_t left = item / NG / pool.kv_heads;                     // the call's block, counted over its requests
  const int h = static_cast<int>(item / NG - left * pool.kv_heads);
  if (left >= most_blocks(kb)) {
    if (left == most_blocks(kb) && item % (NG * pool.kv_heads) == 0) kv_report(kb, pool.page_blocks, err);
    return;
  }
  int b;
  const KvRequest rq = locate_block(kb, pool.page_blocks, left, b);
  if (b < 0) return;
  const int64_t from = rq.L > rq.T ? rq.L - rq.T : 0, blk_at = from / kKvBlock + left;
  uint8_t* blk = kv_block_ptr(pool, kb, D, b, h, blk_at);
  if (blk == nullptr) {
    if (lane == 0) atomicOr(err, kErrIndex);
    return;
  }
  const int t = lane >> 1, g = 2 * pair + (lane & 1);
  const int64_t pos = blk_at * kKvBlock + t;
  const bool mine = pos >= from && pos < rq.L;
  const int64_t tok = rq.q0 + pos - (rq.L - rq.T);
  const uint16_t* src = (which ? v : k) + (mine ? tok : rq.q0) * stride + static_cast<int64_t>(h) * D + 32 * g;
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = mine ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0, 0, 0, 0);
    w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
  }
  float lo = bf16_bits_to_f32(w[0] & 0xFFFF), hi = lo;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float x = __uint_as_float(w[j] << 16), y = __uint_as_float(w[j] & 0xFFFF0000u);
    lo = fminf(lo, fminf(x, y));
    hi = fmaxf(hi, fmaxf(x, y));
    bad |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
  }
  keep_group<D>(blk, blk_at * kKvBlock >= from && blk_at * kKvBlock + kKvBlock <= rq.L, mine, t, g, which, false, lo, hi, bad,
                [&](int j) { return j & 1 ? __uint_as_float(w[j >> 1] & 0xFFFF0000u) : __uint_as_float(w[j >> 1] << 16); }, image[warp]);
}

// One warp per (token, HEADS kv heads), which share its look-ups; lane l writes
// channels VPL*l ..  Four heads a warp where that still leaves warps for all SMs
// (3351 tokens of 8 heads: 7.1 us, 10.5 with one), one where latency counts (16 tokens: 2.1 us, 3.0 with four).
template <int D, int HEADS, typename Out>
__global__ void __launch_bounds__(kKvWarps * 32) kv_read_kernel(KvPool pool, KvBatch kb, Out* __restrict__ ko,
                                                               Out* __restrict__ vo, uint32_t* err) {
  constexpr int NG = D / 32, VPL = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kKvWarps + warp;
  const int quads = (pool.kv_heads + HEADS - 1) / HEADS;
  const int64_t tok = item / quads;
  const int h0 = static_cast<int>(item - tok * quads) * HEADS;
  if (tok >= kb.tokens) {
    if (tok == kb.tokens && h0 == 0) kv_report(kb, pool.page_blocks, err);
    return;
  }
  int b;
  const KvRequest rq = kv_locate(kb, pool.page_blocks, tok, b);
  const uint8_t* blk0 = nullptr;                                // of head h0
  int t = 0;
  if (b >= 0) {
    const int64_t pos = rq.L - rq.T + (tok - rq.q0);
    if (rq.ok && pos >= 0) blk0 = kv_block_ptr(pool, kb, D, b, h0, pos / kKvBlock);
    t = static_cast<int>(pos & (kKvBlock - 1));
    if (blk0 == nullptr && (!rq.ok || pos >= 0) && lane == 0) atomicOr(err, kErrIndex);
  }
  const int d0 = VPL * lane, g = d0 / 32;
#pragma unroll
  for (int hh = 0; hh < HEADS; ++hh) {
    if (h0 + hh >= pool.kv_heads) break;
    float x[2][VPL] = {};                                       // tokens that no cache holds read as zero
    if (blk0 != nullptr) {
      const uint8_t* blk = blk0 + static_cast<int64_t>(hh) * pool.page_blocks * kv_block_bytes(D);
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(blk + 16 * D) + t * NG + g;
      const float ks = bf16_bits_to_f32(__ldg(sc)), km = bf16_bits_to_f32(__ldg(sc + D / 2)), vs = bf16_bits_to_f32(__ldg(sc + D));
      const float vm = bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(blk + 19 * D) + g * kKvBlock + t));
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(blk + kv_k_word(D, t, d0 / 8 % 4, g)));
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int d = d0 + j, c = d % 8;                        // channel within the word: nibble c/2 (+4 if odd)
        const int kc = static_cast<int>(w >> (4 * (c >> 1) + 16 * (c & 1)) & 15) - 8;
        const int vc = static_cast<int>(__ldg(blk + kv_v_byte(D, t, d >> 4, d & 7)) >> (4 * (d >> 3 & 1)) & 15) - 8;
        x[0][j] = __fadd_rn(__fmul_rn(static_cast<float>(kc), ks), km);
        x[1][j] = __fadd_rn(__fmul_rn(static_cast<float>(vc), vs), vm);
      }
    }
    const int64_t out = (tok * pool.kv_heads + h0 + hh) * D + d0;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      Out* to = (which ? vo : ko) + out;
      if constexpr (sizeof(Out) == 4) {
#pragma unroll
        for (int j = 0; j < VPL; j += 2) *reinterpret_cast<float2*>(to + j) = make_float2(x[which][j], x[which][j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < VPL; j += 2) *reinterpret_cast<uint32_t*>(to + j) = pack_bf16x2(x[which][j], x[which][j + 1]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(int D, const KvPool& p, const KvBatch& kb, const void* k, const void* v, int64_t stride,
                             uint32_t* err, cudaStream_t s) {
  // Prompts (64 tokens per request and more on average) by blocks, where there are
  // enough of them to fill the GPU: a warp has 16 times the work.  8 heads of 128, by
  // tokens and by blocks: 1 x 512 tokens 4.0 and 4.5 us, 16 x 64 6.2 and 6.3, 1 x 1024
  // 6.5 and 5.4, 16 x 128 10.5 and 7.7, 1 x 4096 18.7 and 12.0; 2 heads of 64, 3 x 1117: 4.8 and 4.3.
  const bool blocks = kb.tokens >= static_cast<int64_t>(64) * kb.batch && kb.tokens * p.kv_heads >= kFullItems;
  const int64_t items = (blocks ? most_blocks(kb) * (D / 32) : kb.tokens) * p.kv_heads;
  const int64_t grid = items / kKvWarps + 1;              // and a warp that reports what is out of range
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const uint16_t *kk = static_cast<const uint16_t*>(k), *vv = static_cast<const uint16_t*>(v);
  const unsigned g = static_cast<unsigned>(grid), n = kKvWarps * 32;
  if (blocks) switch (D) {
      case 64: return launch(kv_append_blocks_kernel<64>, g, n, 0, s, p, kb, kk, vv, stride, err);
      case 128: return launch(kv_append_blocks_kernel<128>, g, n, 0, s, p, kb, kk, vv, stride, err);
      case 256: return launch(kv_append_blocks_kernel<256>, g, n, 0, s, p, kb, kk, vv, stride, err);
      default: return cudaErrorInvalidValue;
    }
  switch (D) {
    case 64: return launch(kv_append_kernel<64>, g, n, 0, s, p, kb, kk, vv, stride, err);
    case 128: return launch(kv_append_kernel<128>, g, n, 0, s, p, kb, kk, vv, stride, err);
    case 256: return launch(kv_append_kernel<256>, g, n, 0, s, p, kb, kk, vv, stride, err);
    default: return cudaErrorInvalidValue;
  }
}

namespace {

template <int D, int HEADS>
cudaError_t launch_read(const KvPool& p, const KvBatch& kb, void* k, void* v, int out_f32, uint32_t* err, cudaStream_t s) {
  const int64_t grid = kb.tokens * ((p.kv_heads + HEADS - 1) / HEADS) / kKvWarps + 1;      // and a warp that reports
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(grid), n = kKvWarps * 32;
  return out_f32 ? launch(kv_read_kernel<D, HEADS, float>, g, n, 0, s, p, kb, static_cast<float*>(k), static_cast<float*>(v), err)
                 : launch(kv_read_kernel<D, HEADS, uint16_t>, g, n, 0, s, p, kb, static_cast<uint16_t*>(k),
                          static_cast<uint16_t*>(v), err);
}

}  // namespace

cudaError_t launch_kv_read(int D, const KvPool& p, const KvBatch& kb, void* k, void* v, int out_f32, uint32_t* err,
                           cudaStream_t s) {
  // four heads a warp share the look-ups where there are enough: 8 heads of 128, one and
  // four: 512 tokens 3.0 and 3.2 us, 1024 4.2 and 3.5, 4096 12.2 and 8.2
  const bool four = kb.tokens * p.kv_heads >= kFullItems;
  switch (D) {
    case 64: return four ? launch_read<64, 4>(p, kb, k, v, out_f32, err, s) : launch_read<64, 1>(p, kb, k, v, out_f32, err, s);
    case 128: return four ? launch_read<128, 4>(p, kb, k, v, out_f32, err, s) : launch_read<128, 1>(p, kb, k, v, out_f32, err, s);
    case 256: return four ? launch_read<256, 4>(p, kb, k, v, out_f32, err, s) : launch_read<256, 1>(p, kb, k, v, out_f32, err, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace q4nx
