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
#include "q4nx_kv.cuh"

namespace q4nx {

namespace {

constexpr int kKvWarps = 8;      // warps per CTA of the append and read kernels
constexpr int64_t kFullItems = 6144;   // (token, head) pairs from which on larger items pay: below, too few warps have work

// clamp(rint((x - m) / s), -8, 7) + 8 with the quotient correctly rounded; `inv` is
// about 1 / s.  The product with it is within 2^-21 of the quotient, relative,
// so where it is at least 2^-13 from a tie both round alike (|quotient| < 2^7
// or the clamp decides); elsewhere, and where 1 / s is no number, the division is done.
__device__ __forceinline__ uint32_t code_of(float x, float m, float s, float inv) {
  const float d = __fsub_rn(x, m);
  const float q = d * inv;
  float c = rintf(q);
  if (!(fabsf(fabsf(q - c) - 0.5f) > 0x1p-13f) || !(fabsf(q) < 128.f)) c = s == 0.f ? 0.f : rintf(__fdiv_rn(d, s));
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(c, -8.f), 7.f)) + 8);
}
// Scale and middle of a group with smallest and largest value lo, hi; `bad`: one is no number.
__device__ __forceinline__ void scale_of(float lo, float hi, bool bad, uint32_t& s_bits, uint32_t& m_bits) {
  s_bits = f32_to_bf16_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
  const float s = bf16_bits_to_f32(s_bits);
  m_bits = f32_to_bf16_bits(__fadd_rn(lo, __fmul_rn(8.0f, s)));
  const float inf = __int_as_float(0x7f800000);
  if (bad || !(fabsf(s) < inf) || !(fabsf(bf16_bits_to_f32(m_bits)) < inf)) s_bits = m_bits = 0x7FC0;
}

// One warp per (token, kv head).  Lane l holds channels VPL*l .. of the head.
template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_append_kernel(KvPool pool, KvBatch kb, const uint16_t* __restrict__ k,
                                                                 const uint16_t* __restrict__ v, int64_t stride,
                                                                 uint32_t* err) {
  constexpr int VPL = D / 32, NG = D / 32, LPG = 32 / VPL;      // values per lane, groups, lanes per group
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
    float lo = x[0], hi = x[0];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
      bad |= !(fabsf(x[j]) < __int_as_float(0x7f800000));
    }
#pragma unroll
    for (int o = 1; o < LPG; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      bad |= __shfl_xor_sync(0xffffffffu, static_cast<int>(bad), o) != 0;
    }
    uint32_t s_bits, m_bits;
    scale_of(lo, hi, bad, s_bits, m_bits);
    const float s = bf16_bits_to_f32(s_bits), m = bf16_bits_to_f32(m_bits), inv = 1.f / s;
    if (lane % LPG == 0) {
      const int g = lane / LPG;
      uint16_t* sc = reinterpret_cast<uint16_t*>(blk + (which ? 18 : 16) * D);
      sc[t * NG + g] = static_cast<uint16_t>(s_bits);
      sc[D / 2 + (which ? g * kKvBlock + t : t * NG + g)] = static_cast<uint16_t>(m_bits);
    }
    __syncwarp();                                               // the codes of K are read out
#pragma unroll
    for (int j = 0; j < VPL; ++j) codes[warp][lane * VPL + j] = static_cast<uint8_t>(code_of(x[j], m, s, inv));
    __syncwarp();
    if (which == 0) {
      if (lane < D / 8) {                                       // channels 8*lane ..: group lane/4, i lane%4
        const uint2 c = *reinterpret_cast<const uint2*>(&codes[warp][8 * lane]);
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t two = (j < 2 ? c.x : c.y) >> (16 * (j & 1));
          w |= (two & 15) << (4 * j) | (two >> 8 & 15) << (4 * j + 16);
        }
        *reinterpret_cast<uint32_t*>(blk + kv_k_word(D, t, lane & 3, lane >> 2)) = w;
      }
    } else {
#pragma unroll
      for (int n = lane; n < D / 2; n += 32) {
        const int mt = n >> 3, r = n & 7;
        blk[kv_v_byte(D, t, mt, r)] = static_cast<uint8_t>(codes[warp][16 * mt + r] | codes[warp][16 * mt + r + 8] << 4);
      }
    }
  }
}

// A request's tokens lie in T/16 + 2 blocks at most.
__host__ __device__ __forceinline__ int64_t most_blocks(const KvBatch& kb) { return kb.tokens / kKvBlock + 2 * kb.batch; }

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
  // the request: 32 at a time, their block counts added up across the lanes
  int b = -1;
  KvRequest rq = {};
  for (int b0 = 0; b0 < kb.batch && b < 0; b0 += 32) {
    const KvRequest r = b0 + lane < kb.batch ? kv_request(kb, pool.page_blocks, b0 + lane) : KvRequest{0, 0, 0, true};
    const int64_t from = r.L > r.T ? r.L - r.T : 0;             // tokens at positions below 0 are not kept
    const int64_t n = r.T > 0 && r.L > from ? (r.L - 1) / kKvBlock - from / kKvBlock + 1 : 0;
    int64_t end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += u;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, left < end);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      b = b0 + src;
      left -= __shfl_sync(0xffffffffu, end - n, src);
      rq.q0 = __shfl_sync(0xffffffffu, r.q0, src);
      rq.T = __shfl_sync(0xffffffffu, r.T, src);
      rq.L = __shfl_sync(0xffffffffu, r.L, src);
    } else {
      left -= __shfl_sync(0xffffffffu, end, 31);
    }
  }
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
  uint32_t s_bits, m_bits;
  scale_of(lo, hi, bad, s_bits, m_bits);
  const float s = bf16_bits_to_f32(s_bits), m = bf16_bits_to_f32(m_bits), inv = 1.f / s;
  uint32_t c[4] = {};                                           // channel 8i + 2j, +1 of the group: nibbles j, j + 4 of c[i]
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t x = code_of(__uint_as_float(w[j] << 16), m, s, inv), y = code_of(__uint_as_float(w[j] & 0xFFFF0000u), m, s, inv);
    c[j >> 2] |= x << (4 * (j & 3)) | y << (4 * (j & 3) + 16);
  }
  uint16_t* sc = reinterpret_cast<uint16_t*>(blk + (which ? 18 : 16) * D);
  if (mine) {
    sc[t * NG + g] = static_cast<uint16_t>(s_bits);
    sc[D / 2 + (which ? g * kKvBlock + t : t * NG + g)] = static_cast<uint16_t>(m_bits);
  }
  if (which == 0) {
    if (mine)
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(blk + kv_k_word(D, t, i, g)) = c[i];
    return;
  }
  // byte (mt, r): channels r and r + 8 of the 16 of tile mt = 2g + m2: words 2*m2, 2*m2 + 1 of c
  const int base = 8 * D + 512 * pair;
#pragma unroll
  for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int at = 4 * (r >> 1) + 16 * (r & 1);
      const uint32_t byte = (c[2 * m2] >> at & 15) | (c[2 * m2 + 1] >> at & 15) << 4;
      image[warp][kv_v_byte(D, t, 2 * g + m2, r) - base] = static_cast<uint8_t>(byte);
    }
  __syncwarp();
  if (blk_at * kKvBlock >= from && blk_at * kKvBlock + kKvBlock <= rq.L) {
    reinterpret_cast<uint4*>(blk + base)[lane] = reinterpret_cast<const uint4*>(image[warp])[lane];
  } else if (mine) {                                            // other tokens' bytes stay as they are
    for (int n = 0; n < 16; ++n) {
      const int at = kv_v_byte(D, t, 2 * g + (n >> 3), n & 7);
      blk[at] = image[warp][at - base];
    }
  }
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

template <typename... P, typename... A>
cudaError_t launch(void (*f)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
  // programmatic dependent launch: the CTAs start while the previous grid
  // drains and wait for it before their first load
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, static_cast<P>(args)...);
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
