// q4nx_attention.cuh -- what the attention kernels share: arguments, numbers,
// the division of the work, the outputs' places.
#pragma once

#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

namespace q4nx {

constexpr float kRefNone = -3.0e38f;             // reference of a row that has seen nothing
constexpr int kUnitCost = 4;                     // what a unit costs besides its steps, in steps
// a unit is cut between CTAs only so many steps from its ends; a step of the
// kernel for many rows takes 2 us, and up to so many come on top of a CTA's share
template <int RB>
constexpr int cut_steps = RB < 128 ? 4 : 2;
// A CTA's least share.  The parts of a unit are joined by one CTA (few rows), so that a
// unit of n steps is cut into 1.7 sqrt(n) parts at most, where joining takes as long as
// they do: one request of 51015 tokens, one kv head of 128 channels (n = 1594) by 266
// CTAs 31 us, by 80 20, by 40 21; 2 kv heads of 32768 by 304 26, by 103 19, by 51 22.
constexpr int kMinCost = kUnitCost + 2;
__device__ __forceinline__ int least_share(int longest) {
  const int x = static_cast<int>(0.6f * sqrtf(static_cast<float>(longest)));
  return x > kMinCost ? x : kMinCost;
}

// A unit that a CTA began and others ended, for the kernel that joins its parts.
struct Joined {
  int64_t q0, row0;
  int h, rows;
  int parts;                // CTAs with a part of it, from this one on; 0: nothing to join
  int pad;
};

struct AttnArgs {
  KvPool pool;
  KvBatch kb;
  const uint16_t* q;
  int64_t q_stride;         // elements between tokens
  int heads, group;         // query heads, query heads per kv head
  float scale_log2;         // softmax scale * log2(e)
  int64_t window;           // 0: none
  void* out;                // [tokens][heads][D]
  float* lse;               // [tokens][heads] or NULL
  uint32_t* err;
  uint32_t* counters;       // [kKvMaxCtas], zero between calls
  float* partial;           // [2*grid][RB][D + 2]: a CTA's parts of the unit it began and the one it ended with
  Joined* joined;           // [grid], the kernel for many rows
  float* stash;             // [grid][kWarps][RB*D]: a warp's part of the unit it began with
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// d = a b + c, m16n8k16, binary32 sums
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, float c0, float c1, float c2, float c3) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <bool F16>
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  mma<F16>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
// the exact reciprocal of a power of two between 2^-126 and 2^126
__device__ __forceinline__ float inv_pow2(float f) { return __uint_as_float((254u << 23) - __float_as_uint(f)); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// N 32-bit words from shared memory (N = 1, 2 or 4).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (N == 2) {
    const uint2 v = lds64(addr);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = lds128(addr);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {   // of numbers >= 0; short where they are
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// How the steps of all units are divided: position x is step x - start of a
// unit; the units of request b begin at position prefix[b], and the costs
// before them add up to cost[b].
struct Plan {
  const int64_t *prefix, *cost;    // shared memory, [batch + 1]
  int64_t total;                   // of the costs
  int ctas;
  int batch;
};

struct Unit {
  int b, h;
  int64_t rg;               // group of RB query rows
  int64_t start, n;         // first position, number of steps
  int64_t cost;             // the cost before it
  int64_t first;            // first step of the request that any row sees
  KvRequest rq;
};

// First position that some row of the request sees: pages before it need not be there.
__device__ __forceinline__ int64_t first_visible(const KvRequest& rq, int64_t window) {
  if (window <= 0) return 0;
  const int64_t f = rq.L - rq.T + 1 - window;
  return f > 0 ? f : 0;
}
template <int SB>
__device__ __forceinline__ int64_t first_visible_step(const KvRequest& rq, int64_t window) {
  return first_visible(rq, window) / (SB * kKvBlock);
}
template <int SB>
__device__ __forceinline__ int64_t unit_steps(const KvRequest& rq, int64_t window) {
  constexpr int kStepTokens = SB * kKvBlock;
  const int64_t n = (rq.L + kStepTokens - 1) / kStepTokens - first_visible_step<SB>(rq, window);
  return n > 0 ? n : 1;     // an empty request's rows are written too
}

// Steps are of SB 16-token blocks, units of RB query rows.  The unit that holds position x, or (by_cost) the one whose cost range holds x.
template <int SB, int RB>
__device__ __forceinline__ Unit find_unit(const AttnArgs& a, const Plan& pl, int64_t x, bool by_cost = false) {
  const int64_t* at = by_cost ? pl.cost : pl.prefix;
  int lo = 0, hi = pl.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid;
  }
  Unit u;
  u.b = lo;
  u.rq = kv_request(a.kb, a.pool.page_blocks, lo);
  u.n = unit_steps<SB>(u.rq, a.window);
  u.first = first_visible_step<SB>(u.rq, a.window);
  const int64_t groups = quot(u.rq.T * a.group + RB - 1, RB);
  const int64_t k = quot(x - at[lo], by_cost ? u.n + kUnitCost : u.n);
  u.h = static_cast<int>(quot(k, groups));
  u.rg = k - u.h * groups;
  u.start = pl.prefix[lo] + k * u.n;
  u.cost = pl.cost[lo] + k * (u.n + kUnitCost);
  return u;
}

// First position of CTA c: where its share of the costs begins, moved to the
// end of a unit that it falls into less than kCutSteps from.
template <int SB, int RB>
__device__ int64_t bound(const AttnArgs& a, const Plan& pl, int c) {
  if (c >= pl.ctas) return pl.prefix[pl.batch];
  const int64_t q = quot(pl.total, pl.ctas), rest = pl.total - q * pl.ctas;
  const int64_t x = q * c + (c < rest ? c : rest);
  const Unit u = find_unit<SB, RB>(a, pl, x, true);
  const int64_t in = x - u.cost - kUnitCost;
  return u.start + (in < cut_steps<RB> && in < u.n - cut_steps<RB> + 1 ? 0 : in > u.n - cut_steps<RB> ? u.n : in);
}
// The CTA whose share of the costs holds x.
__device__ __forceinline__ int share_of(const Plan& pl, int64_t x) {
  const int64_t q = quot(pl.total, pl.ctas), rest = pl.total - q * pl.ctas;
  return static_cast<int>(x < (q + 1) * rest ? quot(x, q + 1) : rest + quot(x - (q + 1) * rest, q));
}

// Row `row` of request (q0), kv head h: its place among the outputs' rows.
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, int64_t q0, int h, int64_t row) {
  const int64_t tq = quot(row, a.group);
  return (q0 + tq) * a.heads + h * a.group + (row - tq * a.group);
}
template <typename Out>
__device__ __forceinline__ void put(const AttnArgs& a, int64_t at, float y) {
  if constexpr (sizeof(Out) == 4) static_cast<float*>(a.out)[at] = y;
  else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_bits(y);
}
__device__ __forceinline__ float log_total(float m, float l) {
  return l == 0.f ? -__int_as_float(0x7f800000) : (m + lg2(l)) * 0.693147180559945f;
}

// The plan of the call's units, by all threads of a CTA: prefix and cost are
// [batch + 1] and longest is [32] in shared memory.
template <int SB, int RB>
__device__ __forceinline__ Plan make_plan(const AttnArgs& a, int64_t* prefix, int64_t* cost, int* longest) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) prefix[0] = cost[0] = 0;
  // the requests' steps and costs, and their prefix sums
  const int B = a.kb.batch;
  int most = 0;
  for (int b = tid; b < B; b += blockDim.x) {
    const KvRequest rq = kv_request(a.kb, a.pool.page_blocks, b);
    if (!rq.ok && blockIdx.x == 0) atomicOr(a.err, kErrIndex);
    const int64_t units = rq.T > 0 ? quot(rq.T * a.group + RB - 1, RB) * a.pool.kv_heads : 0, n = unit_steps<SB>(rq, a.window);
    prefix[b + 1] = units * n;
    cost[b + 1] = units * (n + kUnitCost);
    if (units > 0) most = max(most, static_cast<int>(n < (1 << 30) ? n : 1 << 30));
  }
  if constexpr (RB < 128) {
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) longest[warp] = most;
  }
  __syncthreads();
  if (warp < 2) {
    int64_t *sum = warp ? cost : prefix, run = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int64_t v = b0 + lane < B ? sum[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      v += run;
      if (b0 + lane < B) sum[b0 + lane + 1] = v;
      run = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  Plan pl;
  pl.prefix = prefix;
  pl.cost = cost;
  pl.batch = B;
  pl.total = cost[B];
  int64_t want = pl.total / kMinCost;
  if constexpr (RB < 128) want = quot(pl.total, least_share(__reduce_max_sync(0xffffffffu, lane < blockDim.x / 32 ? longest[lane] : 0)));
  pl.ctas = want < 1 ? 1 : want < gridDim.x ? static_cast<int>(want) : gridDim.x;
  return pl;
}

// Many query rows per request (q4nx_attention_block.cu; 64 or 128 channels): the
// size of the parts (0 for other sizes), and the launch.
uint64_t attention_block_bytes(int D);
cudaError_t launch_attention_block(int D, const AttnArgs& a, int out_f32, const DeviceInfo& info, cudaStream_t s);

}  // namespace q4nx
