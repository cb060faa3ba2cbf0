// q4nx_kv_store.cuh -- values into the blocks of the 4-bit cache (layout and value
// formula: q4nx_kv.cuh), shared by the append kernels with and without a position rotation.
#pragma once

#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

namespace q4nx {

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
// The range is divided by 15; that of turned keys is multiplied by the 32-bit number nearest to 1/15, one
// operation, whose scale is a bf16 step from the quotient's in one group of 90000 (5 million of turned normal numbers).
__device__ __forceinline__ void scale_of(float lo, float hi, bool bad, bool turned, uint32_t& s_bits, uint32_t& m_bits) {
  const float range = __fsub_rn(hi, lo);
  s_bits = f32_to_bf16_bits(turned ? __fmul_rn(range, 1.0f / 15.0f) : __fdiv_rn(range, 15.0f));
  const float s = bf16_bits_to_f32(s_bits);
  m_bits = f32_to_bf16_bits(__fadd_rn(lo, __fmul_rn(8.0f, s)));
  const float inf = __int_as_float(0x7f800000);
  if (bad || !(fabsf(s) < inf) || !(fabsf(bf16_bits_to_f32(m_bits)) < inf)) s_bits = m_bits = 0x7FC0;
}

// One token's keys (which 0) or values (1) of a head into its block: by a warp, lane l
// with channels VPL*l .. of it; `codes` is the warp's.  turned: see scale_of.
template <int D>
__device__ __forceinline__ void keep_token(uint8_t* blk, int t, int which, bool turned, const float (&x)[D / 32], uint8_t (&codes)[D]) {
  constexpr int VPL = D / 32, NG = D / 32, LPG = 32 / VPL;      // values per lane, groups, lanes per group
  const int lane = threadIdx.x & 31;
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
  scale_of(lo, hi, bad, turned, s_bits, m_bits);
  const float s = bf16_bits_to_f32(s_bits), m = bf16_bits_to_f32(m_bits), inv = 1.f / s;
  if (lane % LPG == 0) {
    const int g = lane / LPG;
    uint16_t* sc = reinterpret_cast<uint16_t*>(blk + (which ? 18 : 16) * D);
    sc[t * NG + g] = static_cast<uint16_t>(s_bits);
    sc[D / 2 + (which ? g * kKvBlock + t : t * NG + g)] = static_cast<uint16_t>(m_bits);
  }
  __syncwarp();                                               // the codes of K are read out
#pragma unroll
  for (int j = 0; j < VPL; ++j) codes[lane * VPL + j] = static_cast<uint8_t>(code_of(x[j], m, s, inv));
  __syncwarp();
  if (which == 0) {
    if (lane < D / 8) {                                       // channels 8*lane ..: group lane/4, i lane%4
      const uint2 c = *reinterpret_cast<const uint2*>(&codes[8 * lane]);
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
      blk[kv_v_byte(D, t, mt, r)] = static_cast<uint8_t>(codes[16 * mt + r] | codes[16 * mt + r + 8] << 4);
    }
  }
}

// A request's tokens lie in T/16 + 2 blocks at most.
__host__ __device__ __forceinline__ int64_t most_blocks(const KvBatch& kb) { return kb.tokens / kKvBlock + 2 * kb.batch; }

// The request of the call's block `left`, counted over its requests' blocks, which
// becomes the request's; by a whole warp, 32 requests at a time, their block counts added up
// across the lanes.  b -1: there is none.
__device__ __forceinline__ KvRequest locate_block(const KvBatch& kb, int page_blocks, int64_t& left, int& b) {
  const int lane = threadIdx.x & 31;
  b = -1;
  KvRequest rq = {};
  for (int b0 = 0; b0 < kb.batch && b < 0; b0 += 32) {
    const KvRequest r = b0 + lane < kb.batch ? kv_request(kb, page_blocks, b0 + lane) : KvRequest{0, 0, 0, true};
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
  return rq;
}

// One group g of token t of a block, keys or values, by a lane: x(j) its values, lo and hi
// their extremes, bad: one is no number.  The warp's lanes 2t + e hold two groups of
// every token, for values neighbouring ones (`image`: the warp's place to gather their bytes).
// mine: the token is the call's; whole: all 16 are; turned: see scale_of.
template <int D, typename X>
__device__ __forceinline__ void keep_group(uint8_t* blk, bool whole, bool mine, int t, int g, int which, bool turned, float lo, float hi, bool bad,
                                           X x, uint8_t (&image)[512]) {
  constexpr int NG = D / 32;
  const int lane = threadIdx.x & 31;
  uint32_t s_bits, m_bits;
  scale_of(lo, hi, bad, turned, s_bits, m_bits);
  const float s = bf16_bits_to_f32(s_bits), m = bf16_bits_to_f32(m_bits), inv = 1.f / s;
  uint32_t c[4] = {};                                           // channel 8i + 2j, +1 of the group: nibbles j, j + 4 of c[i]
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t lo4 = code_of(x(2 * j), m, s, inv), hi4 = code_of(x(2 * j + 1), m, s, inv);
    c[j >> 2] |= lo4 << (4 * (j & 3)) | hi4 << (4 * (j & 3) + 16);
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
  const int base = 8 * D + 512 * (g >> 1);
#pragma unroll
  for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int at = 4 * (r >> 1) + 16 * (r & 1);
      const uint32_t byte = (c[2 * m2] >> at & 15) | (c[2 * m2 + 1] >> at & 15) << 4;
      image[kv_v_byte(D, t, 2 * g + m2, r) - base] = static_cast<uint8_t>(byte);
    }
  __syncwarp();
  if (whole) {
    reinterpret_cast<uint4*>(blk + base)[lane] = reinterpret_cast<const uint4*>(image)[lane];
  } else if (mine) {                                            // other tokens' bytes stay as they are
    for (int n = 0; n < 16; ++n) {
      const int at = kv_v_byte(D, t, 2 * g + (n >> 3), n & 7);
      blk[at] = image[at - base];
    }
  }
}

template <typename... P, typename... A>
inline cudaError_t launch(void (*f)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
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

}  // namespace q4nx
