// q4nx_lora.cu -- the low-rank parts of q4nx_gemm_lora:
//   Y[m] = W x_m + s[id_m] * B[id_m] (A[id_m] x_m),   id_m < 0: W x_m alone.
// Two kernels around the product with W: `shrink` forms t_m = s * A x_m
// (binary32, [64][rank]), `expand` adds B t_m to the product's binary32 output
// and rounds once.  Both are bound by the adapters' bytes when the requests
// use many (64 adapters of rank 16 at 12288 x 4096: 34 MB beside 31 MB of W),
// so each reads an adapter once per launch however many tokens use it.
#include <cooperative_groups.h>

#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

namespace cg = cooperative_groups;

namespace q4nx {

namespace {

constexpr int kMaxTokens = 64;

struct LoraArgs {
  const uint16_t* x;        // [M][K]
  const uint16_t* a;        // [count][R][K]
  const uint16_t* b;        // [count][N][R]
  const float* scale;       // [count]
  const int32_t* ids;       // [M]
  float* t;                 // [64][R]
  const float* base;        // [M][N]
  void* y;                  // [M][N]
  uint32_t* err;
  int64_t K, N;
  int M, R, count;
};

// A token's adapter, -1 for none; one outside the pool is reported and adds nothing.
__device__ __forceinline__ int adapter_of(const LoraArgs& p, int m) {
  if (m >= p.M) return -1;
  const int id = p.ids[m];
  if (id >= p.count) {
    atomicOr(p.err, kErrIndex);
    return -1;
  }
  return id < 0 ? -1 : id;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// t = s * A x of every token of one adapter, 16 rows of A: a cluster of 8 CTAs
// of 8 warps divides the columns in steps of 32 (lane 4n + i of a step holds
// columns 8i..8i+7 of A's rows n, n + 8 and of token n: two k16 products, the
// columns in the same order on both sides, every load 16 bytes).  The warps' sums meet in
// shared memory and the CTAs' through distributed shared memory, in a fixed
// order.  Grid: (8, rank/16, M); a cluster whose token is not the first of its
// adapter has nothing to do.
constexpr int kShrinkCluster = 8, kShrinkWarps = 8;

__global__ void __cluster_dims__(kShrinkCluster, 1, 1) __launch_bounds__(kShrinkWarps * 32)
    lora_shrink_kernel(const LoraArgs p) {
  __shared__ int ids[kMaxTokens], list[kMaxTokens];
  __shared__ int count;
  __shared__ float part[kShrinkWarps][16][kMaxTokens + 1];
  __shared__ float cta[16][kMaxTokens];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster.block_rank());
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < kMaxTokens) ids[tid] = adapter_of(p, tid);
  __syncthreads();
  const int u = blockIdx.z, id = ids[u];
  bool first = id >= 0;
  for (int m = 0; m < u; ++m) first &= ids[m] != id;
  if (!first) return;                                    // the whole cluster alike
  if (tid == 0) {
    int n = 0;
    for (int m = u; m < p.M; ++m)
      if (ids[m] == id) list[n++] = m;
    count = n;
  }
  __syncthreads();
  const int n = count, tiles = (n + 7) / 8;
  const int i = lane & 3, q = lane >> 2, r0 = blockIdx.y * 16;
  const bool row1 = r0 + q + 8 < p.R;                    // rank is a multiple of 8
  const uint16_t* a0 = p.a + (static_cast<int64_t>(id) * p.R + r0 + q) * p.K + 8 * i;
  const uint16_t* a1 = a0 + 8 * p.K;
  float acc[8][4] = {};
  const int64_t steps = p.K / 32, stride = kShrinkCluster * kShrinkWarps;
  for (int64_t s = rank * kShrinkWarps + warp; s < steps; s += stride) {
    const uint4 wa = __ldg(reinterpret_cast<const uint4*>(a0 + 32 * s));
    uint4 wb = make_uint4(0, 0, 0, 0);
    if (row1) wb = __ldg(reinterpret_cast<const uint4*>(a1 + 32 * s));
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= tiles) break;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (8 * t + q < n) x = __ldg(reinterpret_cast<const uint4*>(p.x + list[8 * t + q] * p.K + 32 * s + 8 * i));
      mma_bf16(acc[t], wa.x, wb.x, wa.y, wb.y, x.x, x.y);
      mma_bf16(acc[t], wa.z, wb.z, wa.w, wb.w, x.z, x.w);
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t >= tiles) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][q + 8 * (e >> 1)][8 * t + 2 * i + (e & 1)] = acc[t][e];
  }
  __syncthreads();
  for (int e = tid; e < 16 * n; e += kShrinkWarps * 32) {
    const int r = e / n, m = e - r * n;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kShrinkWarps; ++w) v += part[w][r][m];
    cta[r][m] = v;
  }
  cluster.sync();
  const float sc = p.scale[id];
  for (int e = rank * kShrinkWarps * 32 + tid; e < 16 * n; e += kShrinkCluster * kShrinkWarps * 32) {
    const int r = e / n, m = e - r * n;
    float v = 0.f;
#pragma unroll
    for (int c = 0; c < kShrinkCluster; ++c) v += cluster.map_shared_rank(&cta[0][0], c)[r * kMaxTokens + m];
    if (r0 + r < p.R) p.t[list[m] * p.R + r0 + r] = sc * v;
  }
  cluster.sync();                                        // peers keep their shared memory until all have read
}

// Y = base + B t.  A thread owns one output column n, a CTA kExpandCols
// columns and kExpandTokens tokens taken in the order of their adapters, so
// that a thread reloads its row of B only when the adapter changes.
constexpr int kExpandCols = 128, kExpandTokens = 4;

template <int R, typename Out>
__global__ void __launch_bounds__(kExpandCols) lora_expand_kernel(const LoraArgs p) {
  __shared__ int ids[kMaxTokens], order[kMaxTokens];
  __shared__ __align__(16) float t[kExpandTokens][R];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < kMaxTokens) ids[tid] = adapter_of(p, tid);
  __syncthreads();
  if (tid < p.M) {
    int at = 0;
    for (int m = 0; m < p.M; ++m) at += ids[m] < ids[tid] || (ids[m] == ids[tid] && m < tid);
    order[at] = tid;
  }
  __syncthreads();
  const int m0 = blockIdx.y * kExpandTokens;
  const int tokens = p.M - m0 < kExpandTokens ? p.M - m0 : kExpandTokens;
  for (int e = tid; e < tokens * R; e += kExpandCols) {
    const int j = e / R, m = order[m0 + j];
    t[j][e - j * R] = ids[m] >= 0 ? p.t[m * R + (e - j * R)] : 0.f;
  }
  __syncthreads();
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kExpandCols + tid;
  if (n >= p.N) return;
  int held = -1;
  uint4 w[R / 8];
#pragma unroll
  for (int j = 0; j < kExpandTokens; ++j) {
    if (j >= tokens) break;
    const int m = order[m0 + j], id = ids[m];
    float y = p.base[m * p.N + n];
    if (id >= 0) {
      if (id != held) {
        const uint4* src = reinterpret_cast<const uint4*>(p.b + (static_cast<int64_t>(id) * p.N + n) * R);
#pragma unroll
        for (int c = 0; c < R / 8; ++c) w[c] = __ldg(src + c);
        held = id;
      }
      float add = 0.f;
#pragma unroll
      for (int c = 0; c < R / 8; ++c) {
        const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          add = fmaf(__uint_as_float(v[k] << 16), t[j][8 * c + 2 * k], add);
          add = fmaf(__uint_as_float(v[k] & 0xFFFF0000u), t[j][8 * c + 2 * k + 1], add);
        }
      }
      y += add;
    }
    if constexpr (sizeof(Out) == 4) static_cast<float*>(p.y)[m * p.N + n] = y;
    else static_cast<uint16_t*>(p.y)[m * p.N + n] = f32_to_bf16_bits(y);
  }
}

template <typename Out>
cudaError_t launch_expand(const LoraArgs& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + kExpandCols - 1) / kExpandCols),
                     static_cast<unsigned>((p.M + kExpandTokens - 1) / kExpandTokens));
  cfg.blockDim = dim3(kExpandCols);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (p.R) {
    case 8: return cudaLaunchKernelEx(&cfg, lora_expand_kernel<8, Out>, p);
    case 16: return cudaLaunchKernelEx(&cfg, lora_expand_kernel<16, Out>, p);
    case 32: return cudaLaunchKernelEx(&cfg, lora_expand_kernel<32, Out>, p);
    case 64: return cudaLaunchKernelEx(&cfg, lora_expand_kernel<64, Out>, p);
    case 128: return cudaLaunchKernelEx(&cfg, lora_expand_kernel<128, Out>, p);
    default: return cudaErrorInvalidValue;
  }
}

LoraArgs lora_args(const LoraCall& c) {
  LoraArgs p;
  p.x = static_cast<const uint16_t*>(c.x);
  p.a = static_cast<const uint16_t*>(c.a);
  p.b = static_cast<const uint16_t*>(c.b);
  p.scale = c.scale;
  p.ids = c.ids;
  p.t = c.t;
  p.base = c.base;
  p.y = c.y;
  p.err = c.err;
  p.K = c.K;
  p.N = c.N;
  p.M = c.M;
  p.R = c.R;
  p.count = c.count;
  return p;
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraCall& c, cudaStream_t s) {
  const LoraArgs p = lora_args(c);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kShrinkCluster, static_cast<unsigned>((p.R + 15) / 16), static_cast<unsigned>(p.M));
  cfg.blockDim = dim3(kShrinkWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_shrink_kernel, p);
}

cudaError_t launch_lora_expand(const LoraCall& c, int out_f32, cudaStream_t s) {
  const LoraArgs p = lora_args(c);
  return out_f32 ? launch_expand<float>(p, s) : launch_expand<uint16_t>(p, s);
}

}  // namespace q4nx
