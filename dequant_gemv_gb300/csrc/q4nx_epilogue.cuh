// q4nx_epilogue.cuh -- what q4nx_gemm_epilogue does to a product before its one
// rounding, shared by the GEMV and GEMM kernels:
//   y = act(acc + bias[n]) * mul[m][n] + residual[m][n],
// each step in binary32.  An element's operands are read by the CTA that stores it,
// before it does, so that mul or residual may be the output itself.
//
// What it costs (back to back in a graph): 1024x2048 q4_1, one token with a residual 4.6 -> 5.1 us; 12288x4096 q4_1, one
// token, SiLU and gate 10.4 -> 11.0, 64 tokens 14.0 -> 16.4, which moves 1.6 MB more and the activation's instructions at
// the launch's end, 12 warps of an SM on 128 rows x 64 tokens; Q8 4096x12288, 33 tokens, bias, GELU (tanh) and
// residual 17.6 -> 21.4 (whole calls 22.7).  The tensor-core kernel spills with an epilogue (216 bytes of stores, 496 of
// loads at 128 registers, none without).  As operations of their own behind the product these read and write it again.
#pragma once

#include <cstdint>

#include "q4nx_device.cuh"

namespace q4nx {

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct Epilogue {
  const uint16_t* bias = nullptr;      // bf16 [N]
  const uint16_t* mul = nullptr;       // bf16 [M][N], mul_stride elements from token to token
  const uint16_t* residual = nullptr;  // bf16 [M][N]
  int64_t mul_stride = 0, residual_stride = 0;
  int act = kActNone;
};

// x / (1 + exp(-z)), right to a few units in the last place down to z = -87, where the denominator is still
// below 2^126 and its reciprocal normal.  Further on that ends, and then binary32, while the quotient
// is a normal number down to -92: far_tail.
constexpr float kFarTail = -87.f;
__device__ __forceinline__ float times_sigmoid(float x, float z) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + expf(-z)));
  return x * y;
}
// That, for z below kFarTail: x exp(z), the power taken by halves, which stay normal (IEEE arithmetic's NaN where both are infinite).
__device__ __forceinline__ float far_tail(float x, float z) {
  const float half = expf(0.5f * z);
  return x * half * half;
}
// 2 u for tanh GELU: 0.5 x (1 + tanh u) = x / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3)
__device__ __forceinline__ float gelu_tanh_z(float x) { return 1.5957691216057308f * fmaf(0.044715f * x * x, x, x); }

template <int ACT>
__device__ __forceinline__ float activated(float x) {
  if constexpr (ACT == kActRelu) return x < 0.f ? 0.f : x;                       // NaN stays NaN
  // erfc, not 1 + erf: that would leave nothing of the tail below -4
  if constexpr (ACT == kActGelu) return 0.5f * x * erfcf(-0.70710678118654752f * x);
  return x;
}

// Four at a call: its code, the longest of them, is there once and warm from the second call on.
static __device__ __noinline__ float4 gelu4(float4 x) {
  return make_float4(activated<kActGelu>(x.x), activated<kActGelu>(x.y), activated<kActGelu>(x.z), activated<kActGelu>(x.w));
}

// Both kinds of x / (1 + exp(-z)), T at a time.  The tail's test is one for all of them: a branch for each
// kept them from running side by side (12288x4096, 64 tokens, SiLU and gate 17.4 us; this way 16.3, without the tail 16.1).
template <int T, typename Z>
__device__ __forceinline__ void times_sigmoid(float (&v)[T], Z z) {
  float y[T], least = z(v[0]);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    least = fminf(least, z(v[t]));
    y[t] = times_sigmoid(v[t], z(v[t]));
  }
  if (least < kFarTail) {
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (z(v[t]) < kFarTail) y[t] = far_tail(v[t], z(v[t]));
  }
#pragma unroll
  for (int t = 0; t < T; ++t) v[t] = y[t];
}

template <int T>
__device__ __forceinline__ void activate(int act, float (&v)[T]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int t = 0; t < T; ++t) v[t] = activated<kActRelu>(v[t]);
      break;
    case kActGelu:
      if constexpr (T % 4 == 0) {
#pragma unroll
        for (int t = 0; t < T; t += 4) {
          const float4 y = gelu4(make_float4(v[t], v[t + 1], v[t + 2], v[t + 3]));
          v[t] = y.x, v[t + 1] = y.y, v[t + 2] = y.z, v[t + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int t = 0; t < T; ++t) v[t] = activated<kActGelu>(v[t]);
      }
      break;
    case kActGeluTanh: times_sigmoid(v, [](float x) { return gelu_tanh_z(x); }); break;
    case kActSilu: times_sigmoid(v, [](float x) { return x; }); break;
    default: break;
  }
}

// One element, its operands straight from memory.
__device__ __forceinline__ float epilogue_of(const Epilogue& e, int64_t n, int m, float acc) {
  const uint32_t b = e.bias != nullptr ? e.bias[n] : 0u, g = e.mul != nullptr ? e.mul[m * e.mul_stride + n] : 0u,
                 r = e.residual != nullptr ? e.residual[m * e.residual_stride + n] : 0u;
  float v[1] = {e.bias != nullptr ? acc + bf16_bits_to_f32(b) : acc};
  activate<1>(e.act, v);
  if (e.mul != nullptr) v[0] *= bf16_bits_to_f32(g);
  if (e.residual != nullptr) v[0] += bf16_bits_to_f32(r);
  return v[0];
}

}  // namespace q4nx
