// q4nx_lora.cu -- the low-rank parts of q4nx_gemm_lora:
//   Y[m] = W x_m + s[id_m] * B[id_m] (A[id_m] x_m),   id_m < 0: W x_m alone.
// Two kernels around the product with W: `shrink` forms t_m = s * A x_m
// (binary32, [64][rank]), `expand` adds B t_m to the product's binary32 output
// and rounds once.  Both are bound by the adapters' bytes when the requests use many (64 adapters of rank 16 at
// 12288 x 4096: 34 MB beside 31 MB of W), and by latency otherwise: each
// issues all loads of a step before the first product.
//
// Behind the tensor-core product, whose 96 or 128 CTAs leave SMs free, shrink runs
// beside it: the product lets it start once its own wait for earlier grids is over (cold
// L2, the whole call: 64 adapters of rank 16 at 12288 x 4096 34.0 -> 27.9 us; rank 64 at
// 4096 x 12288, 64 tokens of one adapter 42.2 -> 36.0).  Bringing the used adapters' B
// to L2 in that time takes bandwidth from the product: 0.4 to 2 us gained with 13 to 25 MB
// of them at 12288 x 4096, 2 to 15 lost with 0.5 MB at 4096 x 12288, with 25 MB at 24576 x
// 4096 and with 31 MB and more, so that it is left to `expand`.  `expand` starts when both have
// ended: let start early, its CTAs crowd on the few free SMs (2 to 4 us more).
// The few-token product fills every SM: shrink goes before it there.
#include <algorithm>
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
  float* t;                 // [splits][64][R]
  int2* sorted;             // [M]: the tokens with their adapters, in the order of the adapters
  const float* base;        // [M][N]
  void* y;                  // [M][N]
  uint32_t* err;
  int64_t K, N;
  int M, R, count, splits;
  int beside;               // shrink runs beside the product and ends after it
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

// t = s * A x of every token, in items: one adapter, 16 rows of A, kSplitCols
// columns (or their share, where the columns are cut into kMaxSplits parts,
// which `expand` adds in order).  A cluster of 8 CTAs of 8 warps divides an
// item's columns in steps of 32 (lane 4n + i of a step holds columns
// 8i..8i+7 of A's rows n, n + 8 and of token n: two k16 products, the columns in
// the same order on both sides, every load 16 bytes): two steps a warp, whose loads
// are issued together.  What counts is how many loads the whole GPU has in
// flight: without the parts, at rank 64, 12288 columns (Q8) and 64 tokens of one adapter, only 32
// CTAs have work, and the whole call takes 45 us (cold L2) instead of 37.  With many adapters there
// is work enough and the parts cost instead: 4 of them 39 and 40, 16 of them 45 and 58, 64
// of them 97 and 134.  The warps' sums meet in shared memory and the CTAs'
// through distributed shared memory, in a fixed order.
constexpr int kShrinkWarps = 8, kShrinkCluster = 8, kShrinkPerSm = 3;
constexpr int kSplitCols = 4096, kMaxSplits = 8;

__global__ void __cluster_dims__(kShrinkCluster, 1, 1) __launch_bounds__(kShrinkWarps * 32, kShrinkPerSm) lora_shrink_kernel(const LoraArgs p) {
  __shared__ int ids[kMaxTokens], list[kMaxTokens], lead[kMaxTokens];
  __shared__ uint32_t leads[2];
  __shared__ int count;
  __shared__ float part[kShrinkWarps][16][kMaxTokens + 1];
  __shared__ float sum[kMaxTokens][16];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!p.beside) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  if (tid < kMaxTokens) ids[tid] = adapter_of(p, tid);
  __syncthreads();
  if (tid < kMaxTokens) {                                  // the first token of each adapter, in order
    const int id = ids[tid];
    bool first = id >= 0;
#pragma unroll 8
    for (int m = 0; m < kMaxTokens; ++m) first &= m >= tid || ids[m] != id;
    const uint32_t b = __ballot_sync(0xffffffffu, first);
    if (lane == 0) leads[warp] = b;
    __syncwarp();
  }
  __syncthreads();
  if (tid < kMaxTokens && (leads[warp] >> lane & 1))
    lead[(warp ? __popc(leads[0]) : 0) + __popc(leads[warp] & ((1u << lane) - 1))] = tid;
  if (blockIdx.x == 0 && tid < p.M) {                       // for `expand`
    int at = 0;
    const int id = ids[tid];
#pragma unroll 8
    for (int m = 0; m < kMaxTokens; ++m) at += m < p.M && (ids[m] < id || (ids[m] == id && m < tid));
    p.sorted[at] = make_int2(tid, id);
  }
  const int adapters = __popc(leads[0]) + __popc(leads[1]), tiles_r = (p.R + 15) / 16;
  const int items = adapters * tiles_r * p.splits;
  const int i = lane & 3, q = lane >> 2;
  const int64_t steps = p.K / 32;
#pragma unroll 1
  for (int item = blockIdx.x / kShrinkCluster; item < items; item += gridDim.x / kShrinkCluster) {      // the whole cluster alike
    const int split = item % p.splits, r0 = item / p.splits % tiles_r * 16;
    __syncthreads();                                       // lead is written; the last item's list and part are read
    const int u = lead[item / p.splits / tiles_r], id = ids[u];
    if (warp < 2) {                                        // its tokens, in order
      const uint32_t lo = __ballot_sync(0xffffffffu, ids[lane] == id), hi = __ballot_sync(0xffffffffu, ids[lane + 32] == id);
      const uint32_t mine = warp ? hi : lo;
      if (mine >> lane & 1) list[(warp ? __popc(lo) : 0) + __popc(mine & ((1u << lane) - 1))] = tid;
      if (tid == 0) count = __popc(lo) + __popc(hi);
    }
    __syncthreads();
    const int n = count, tiles = (n + 7) / 8;
    const bool row1 = r0 + q + 8 < p.R;                    // rank is a multiple of 8
    const uint16_t* a0 = p.a + (static_cast<int64_t>(id) * p.R + r0 + q) * p.K + 8 * i;
    float acc[8][4] = {};
    constexpr int kStride = kShrinkCluster * kShrinkWarps;
    const int64_t s1 = steps * (split + 1) / p.splits;
    for (int64_t s = steps * split / p.splits + rank * kShrinkWarps + warp; s < s1; s += 2 * kStride) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const bool two = s + kStride < s1;
      uint4 wa[2], wb[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint16_t* at = a0 + 32 * (s + k * kStride);
        wa[k] = k == 0 || two ? __ldg(reinterpret_cast<const uint4*>(at)) : zero;
        wb[k] = row1 && (k == 0 || two) ? __ldg(reinterpret_cast<const uint4*>(at + 8 * p.K)) : zero;
      }
#pragma unroll
      for (int t0 = 0; t0 < 8; t0 += 2) {
        if (t0 >= tiles) break;
        uint4 x[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int m = 8 * (t0 + t) + q;
          const uint16_t* at = p.x + static_cast<int64_t>(list[m < n ? m : 0]) * p.K + 32 * s + 8 * i;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            x[t][k] = m < n && (k == 0 || two) ? __ldg(reinterpret_cast<const uint4*>(at + 32 * kStride * k)) : zero;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mma_bf16(acc[t0 + t], wa[k].x, wb[k].x, wa[k].y, wb[k].y, x[t][k].x, x[t][k].y);
            mma_bf16(acc[t0 + t], wa[k].z, wb[k].z, wa[k].w, wb[k].w, x[t][k].z, x[t][k].w);
          }
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < tiles) {
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][q + 8 * (e >> 1)][8 * t + 2 * i + (e & 1)] = acc[t][e];
      }
    __syncthreads();
    for (int e = tid; e < 16 * n; e += kShrinkWarps * 32) {
      const int m = e >> 4, r = e & 15;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kShrinkWarps; ++w) v += part[w][r][m];
      sum[m][r] = v;
    }
    cluster.sync();
    const float sc = p.scale[id];
    for (int e = rank * kShrinkWarps * 32 + tid; e < 16 * n; e += kStride * 32) {
      const int m = e >> 4, r = e & 15;
      float v = 0.f;
#pragma unroll
      for (int c = 0; c < kShrinkCluster; ++c) v += cluster.map_shared_rank(&sum[0][0], c)[e];
      if (r0 + r < p.R) p.t[(split * kMaxTokens + list[m]) * p.R + r0 + r] = sc * v;
    }
    cluster.sync();                                        // peers keep their sums until all have read
  }
  // `expand` waits for this grid alone: it has the product when this grid ends after
  // it.  One CTA sees to that, so that the others make room for those still to come.
  if (p.beside && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Y = base + B t.  A thread owns one output column n, a CTA kExpandCols
// columns and kExpandTokens tokens taken in the order of their adapters, so
// that a thread reloads its row of B only when the adapter changes.  Few registers and
// many CTAs keep the loads in flight (all loads of four tokens held at once: 12.6 us
// instead of 9.2 for 64 adapters of rank 16 at 12288 rows, fewer CTAs fit).
constexpr int kExpandCols = 128, kExpandTokens = 4;

template <int R, typename Out>
__global__ void __launch_bounds__(kExpandCols) lora_expand_kernel(const LoraArgs p) {
  __shared__ __align__(16) float t[kExpandTokens][R];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int m0 = blockIdx.y * kExpandTokens;
  const int tokens = p.M - m0 < kExpandTokens ? p.M - m0 : kExpandTokens;
  int2 token[kExpandTokens];                              // (token, adapter)
#pragma unroll
  for (int j = 0; j < kExpandTokens; ++j) token[j] = p.sorted[m0 + (j < tokens ? j : 0)];
#pragma unroll
  for (int j = 0; j < kExpandTokens; ++j)
    for (int r = tid; r < R; r += kExpandCols) {
      float v = 0.f;
      if (token[j].y >= 0)
        for (int c = 0; c < p.splits; ++c) v += p.t[(c * kMaxTokens + token[j].x) * R + r];
      t[j][r] = v;
    }
  __syncthreads();
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kExpandCols + tid;
  if (n >= p.N) return;
  int held = -1;
  uint4 w[R / 8];
#pragma unroll
  for (int j = 0; j < kExpandTokens; ++j) {
    if (j >= tokens) break;
    const int m = token[j].x, id = token[j].y;
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
  p.sorted = reinterpret_cast<int2*>(c.t + static_cast<int64_t>(lora_splits(c.K)) * kMaxTokens * c.R);
  p.base = c.base;
  p.y = c.y;
  p.err = c.err;
  p.K = c.K;
  p.N = c.N;
  p.M = c.M;
  p.R = c.R;
  p.count = c.count;
  p.splits = lora_splits(c.K);
  p.beside = 0;
  return p;
}

}  // namespace

int lora_splits(int64_t K) { return static_cast<int>(std::clamp<int64_t>(K / kSplitCols, 1, kMaxSplits)); }

cudaError_t launch_lora_shrink(const LoraCall& c, const DeviceInfo& info, bool beside, cudaStream_t s) {
  LoraArgs p = lora_args(c);
  p.beside = beside;
  cudaLaunchConfig_t cfg = {};
  // as many clusters as there can be items and as the GPU holds
  const int clusters = std::min(p.M * ((p.R + 15) / 16) * p.splits, std::max(1, kShrinkPerSm * info.sms / kShrinkCluster));
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kShrinkCluster));
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
