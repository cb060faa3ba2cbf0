// q4nx_kv.cu -- new keys and values into the 4-bit cache, and cached ones back
// out of it (layout and value formula: q4nx_kv.cuh).
//
// Quantisation of 32 values x of one token and head, each step one IEEE
// binary32 operation, so that every machine takes the same codes:
//   lo, hi = min, max;  scale = bf16((hi - lo) / 15);  mid = bf16(lo + 8*scale)
//   code = clamp(rint((x - mid) / scale), -8, 7) + 8   (ties to even; 8 where scale is 0)
// A group that holds a NaN or an infinity, or whose range overflows, keeps NaN
// as its scale and mid: all of it reads as NaN.
#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

namespace q4nx {

namespace {

constexpr int kKvWarps = 8;      // warps per CTA of the append and read kernels

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
  if (tok >= kb.tokens) return;
  const int b = kv_find_request(kb, tok);
  if (b < 0) return;                                            // a token of no request
  const KvRequest rq = kv_request(kb, pool.page_blocks, b);
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
    const uint16_t* src = (which ? v : k) + tok * stride + static_cast<int64_t>(h) * D + lane * VPL;
    float x[VPL];
#pragma unroll
    for (int j = 0; j < VPL; j += 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(src + j);
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
    uint32_t s_bits = f32_to_bf16_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = bf16_bits_to_f32(s_bits);
    uint32_t m_bits = f32_to_bf16_bits(__fadd_rn(lo, __fmul_rn(8.0f, s)));
    const float m = bf16_bits_to_f32(m_bits);
    if (bad || !(fabsf(s) < __int_as_float(0x7f800000)) || !(fabsf(m) < __int_as_float(0x7f800000))) s_bits = m_bits = 0x7FC0;
    if (lane % LPG == 0) {
      const int g = lane / LPG;
      uint16_t* sc = reinterpret_cast<uint16_t*>(blk + (which ? 18 : 16) * D);
      sc[t * NG + g] = static_cast<uint16_t>(s_bits);
      sc[D / 2 + (which ? g * kKvBlock + t : t * NG + g)] = static_cast<uint16_t>(m_bits);
    }
    __syncwarp();                                               // the codes of K are read out
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      float c = 0.f;
      if (s != 0.f) c = rintf(__fdiv_rn(__fsub_rn(x[j], m), s));
      c = fminf(fmaxf(c, -8.f), 7.f);
      codes[warp][lane * VPL + j] = static_cast<uint8_t>(static_cast<int>(c) + 8);
    }
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

// One warp per (token, kv head); lane l writes channels l, l+32, ...
template <int D, typename Out>
__global__ void __launch_bounds__(kKvWarps * 32) kv_read_kernel(KvPool pool, KvBatch kb, Out* __restrict__ ko,
                                                               Out* __restrict__ vo, uint32_t* err) {
  constexpr int NG = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kKvWarps + warp;
  const int64_t tok = item / pool.kv_heads;
  const int h = static_cast<int>(item - tok * pool.kv_heads);
  if (tok >= kb.tokens) return;
  const int b = kv_find_request(kb, tok);
  const uint8_t* blk = nullptr;
  int t = 0;
  if (b >= 0) {
    const KvRequest rq = kv_request(kb, pool.page_blocks, b);
    const int64_t pos = rq.L - rq.T + (tok - rq.q0);
    if (rq.ok && pos >= 0) blk = kv_block_ptr(pool, kb, D, b, h, pos / kKvBlock);
    t = static_cast<int>(pos & (kKvBlock - 1));
    if (blk == nullptr && (!rq.ok || pos >= 0) && lane == 0) atomicOr(err, kErrIndex);
  }
  const int64_t out = (tok * pool.kv_heads + h) * D;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int d = g * 32 + lane;
    float kx = 0.f, vx = 0.f;                                   // tokens that no cache holds read as zero
    if (blk != nullptr) {
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(blk + 16 * D) + t * NG + g;
      const uint16_t* vm = reinterpret_cast<const uint16_t*>(blk + 19 * D) + g * kKvBlock + t;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + kv_k_word(D, t, lane >> 3, g));
      const int c = lane & 7;                                   // channel within the word: nibble c/2 (+4 if odd)
      const int kc = static_cast<int>(w >> (4 * (c >> 1) + 16 * (c & 1)) & 15) - 8;
      const int vc = static_cast<int>(blk[kv_v_byte(D, t, d >> 4, d & 7)] >> (4 * (d >> 3 & 1)) & 15) - 8;
      kx = __fadd_rn(__fmul_rn(static_cast<float>(kc), bf16_bits_to_f32(sc[0])), bf16_bits_to_f32(sc[D / 2]));
      vx = __fadd_rn(__fmul_rn(static_cast<float>(vc), bf16_bits_to_f32(sc[D])), bf16_bits_to_f32(*vm));
    }
    if constexpr (sizeof(Out) == 4) {
      ko[out + d] = kx;
      vo[out + d] = vx;
    } else {
      ko[out + d] = f32_to_bf16_bits(kx);
      vo[out + d] = f32_to_bf16_bits(vx);
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
  const int64_t grid = (kb.tokens * p.kv_heads + kKvWarps - 1) / kKvWarps;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const uint16_t *kk = static_cast<const uint16_t*>(k), *vv = static_cast<const uint16_t*>(v);
  const unsigned g = static_cast<unsigned>(grid), n = kKvWarps * 32;
  switch (D) {
    case 64: return launch(kv_append_kernel<64>, g, n, 0, s, p, kb, kk, vv, stride, err);
    case 128: return launch(kv_append_kernel<128>, g, n, 0, s, p, kb, kk, vv, stride, err);
    case 256: return launch(kv_append_kernel<256>, g, n, 0, s, p, kb, kk, vv, stride, err);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv_read(int D, const KvPool& p, const KvBatch& kb, void* k, void* v, int out_f32, uint32_t* err,
                           cudaStream_t s) {
  const int64_t grid = (kb.tokens * p.kv_heads + kKvWarps - 1) / kKvWarps;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(grid), n = kKvWarps * 32;
  float *kf = static_cast<float*>(k), *vf = static_cast<float*>(v);
  uint16_t *kh = static_cast<uint16_t*>(k), *vh = static_cast<uint16_t*>(v);
  switch (D) {
    case 64:
      return out_f32 ? launch(kv_read_kernel<64, float>, g, n, 0, s, p, kb, kf, vf, err)
                     : launch(kv_read_kernel<64, uint16_t>, g, n, 0, s, p, kb, kh, vh, err);
    case 128:
      return out_f32 ? launch(kv_read_kernel<128, float>, g, n, 0, s, p, kb, kf, vf, err)
                     : launch(kv_read_kernel<128, uint16_t>, g, n, 0, s, p, kb, kh, vh, err);
    case 256:
      return out_f32 ? launch(kv_read_kernel<256, float>, g, n, 0, s, p, kb, kf, vf, err)
                     : launch(kv_read_kernel<256, uint16_t>, g, n, 0, s, p, kb, kh, vh, err);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace q4nx
