// q4nx_logprobs.cu -- log-probabilities of rows of logits in one pass:
//   lse = log sum exp x,  lp(token) = x[token] - lse,  H = lse - sum p x,
// and the `top` largest with their indexes (ties: lowest index).
//
// Bound: the logits' bytes, once; at one row, latency.  A cluster of C CTAs
// takes a row; each thread keeps the running maximum m, z = sum exp(x - m) and
// w = sum exp(x - m) (x - m) of its elements, moved to a new maximum once per
// batch of loads (exp of 0 at the maximum, never an overflow; a centred w
// keeps the entropy free of cancellation).
//
// Top alternatives without a second pass over memory: the j-th largest of a
// warp's 32 thread maxima is reached by at least j elements of that warp, so the
// smallest such value over W warps, j = ceil(top / W), is a floor for the CTA's
// top elements.  W counts the warps whose threads have elements (of the last one at
// least half): a floor made by a nearly empty warp lets everything through.  Only threads whose own maximum reaches the
// floor have their elements read again (from L2, by their whole warp; one thread in
// ten), and the elements at or above it, about a hundred, get their ranks by
// counting.  Rows with more than kCand such elements (many equal ones; so few above -inf
// that -inf is the floor) take `top` rounds of "largest below the previous" instead: one
// row of 151936 of which 40 are allowed, top 20, 80 us instead of 10.
#include <cooperative_groups.h>

#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

namespace cg = cooperative_groups;

namespace q4nx {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCand = 1024;          // candidates of a CTA
constexpr int kBatch = 8;            // 16-byte loads a thread has in flight
constexpr int kMaxTop = 32, kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896f;

struct Args {
  const uint8_t* logits;
  int64_t V, pitch;                  // columns, bytes between rows
  const int32_t* tokens;
  float *logprob, *entropy, *lse;
  int32_t* top_idx;
  float* top_lp;
  int top;
};

struct Stat {
  float m, z, w;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
// what is subtracted from x for a running maximum m: a row of -inf alone stays all zeros
__device__ __forceinline__ float shift_of(float m) { return m == neg_inf() ? 0.f : m; }

__device__ __forceinline__ void move_to(Stat& s, float m) {
  const float d = shift_of(s.m) - shift_of(m);         // <= 0 once s holds anything
  const float f = s.z == 0.f ? 0.f : ex2(d * kLog2e);
  s.w = f == 0.f ? 0.f : f * fmaf(s.z, d, s.w);
  s.z *= f;
  s.m = m;
}
// A warp's statistics joined: moved to the largest maximum, then added.
__device__ __forceinline__ Stat join_warp(Stat s) {
  float m = s.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  move_to(s, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
  }
  return s;
}
__device__ __forceinline__ void add(Stat& s, float x, float shift) {
  const float d = x - shift;
  const float e = ex2(d * kLog2e);
  s.z += e;
  s.w = fmaf(e, fmaxf(d, -300.f), s.w);                // e is 0 there, and 0 * -inf is not
}
__device__ __forceinline__ uint32_t ord_of(float v) { return static_cast<uint32_t>(argmax_key(v, 0) >> 32); }
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  if (o == 0xFFFFFFFFu) return __int_as_float(0x7fc00000);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

template <bool BF16>
struct Row {
  static constexpr int VE = BF16 ? 8 : 4;              // elements per 16-byte load
  const uint8_t* p;
  int64_t V;
  int64_t head;                                        // elements before the first 16-byte boundary
  int64_t vecs;                                        // whole 16-byte loads
  int64_t tail;                                        // elements after them
  __device__ Row(const uint8_t* row, int64_t v) : p(row), V(v) {
    const int es = BF16 ? 2 : 4;
    head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / es;
    if (head > V) head = V;
    vecs = (V - head) / VE;
    tail = V - head - vecs * VE;
  }
  __device__ float at(int64_t i) const {
    if constexpr (BF16) return bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(p) + i));
    else return __ldg(reinterpret_cast<const float*>(p) + i);
  }
  __device__ uint4 load(int64_t v) const { return __ldg(reinterpret_cast<const uint4*>(p + head * (BF16 ? 2 : 4)) + v); }
  __device__ static float pick(const uint4& u, int e) {
    const uint32_t w = (e / (VE / 4)) == 0 ? u.x : (e / (VE / 4)) == 1 ? u.y : (e / (VE / 4)) == 2 ? u.z : u.w;
    if constexpr (BF16) return (e & 1) ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
    else return __uint_as_float(w);
  }
};

// The elements of one thread: every kThreads-th load of the CTA's share, and
// (first CTA) one of the row's unaligned ends.
template <bool BF16, typename F>
__device__ __forceinline__ void for_elements(const Row<BF16>& row, int64_t v0, int64_t v1, int64_t end_elem, F f) {
  constexpr int VE = Row<BF16>::VE;
#pragma unroll 1
  for (int64_t v = v0 + threadIdx.x; v < v1; v += kThreads) {
    const uint4 u = row.load(v);
#pragma unroll
    for (int e = 0; e < VE; ++e) f(Row<BF16>::pick(u, e), row.head + v * VE + e);
  }
  if (end_elem >= 0) f(row.at(end_elem), end_elem);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const Args a) {
  constexpr int VE = Row<BF16>::VE;
  __shared__ Stat stats[kWarps];
  __shared__ uint32_t floor_of[kWarps];
  __shared__ uint64_t cand[kCand];
  __shared__ uint64_t best[kMaxTop];                   // this CTA's, largest first
  __shared__ uint64_t all[kMaxTop * kMaxCluster];
  __shared__ uint64_t reduce[kWarps];
  __shared__ int found;
  __shared__ float final_lse;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t m = blockIdx.y;
  const Row<BF16> row(a.logits + m * a.pitch, a.V);
  const int64_t v0 = row.vecs * rank / C, v1 = row.vecs * (rank + 1) / C;
  int64_t end_elem = -1;
  if (rank == 0) {
    if (tid < row.head) end_elem = tid;
    else if (tid - row.head < row.tail) end_elem = row.V - row.tail + (tid - row.head);
  }
  Stat s = {neg_inf(), 0.f, 0.f};
  float big = neg_inf();
  bool any = end_elem >= 0;
  if (any) {
    const float x = row.at(end_elem);
    s.m = big = fmaxf(x, neg_inf());
    add(s, x, shift_of(s.m));
  }
  for (int64_t v = v0 + tid; v < v1; v += kBatch * kThreads) {
    uint4 u[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (v + k * kThreads < v1) u[k] = row.load(v + k * kThreads);
    float mx = s.m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (v + k * kThreads < v1) {
#pragma unroll
        for (int e = 0; e < VE; ++e) mx = fmaxf(mx, Row<BF16>::pick(u[k], e));
      }
    move_to(s, mx);
    const float shift = shift_of(mx);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (v + k * kThreads < v1) {
#pragma unroll
        for (int e = 0; e < VE; ++e) add(s, Row<BF16>::pick(u[k], e), shift);
      }
    big = mx;
    any = true;
  }
  // the largest value of this thread in the order of the top list (NaN above
  // all); a NaN total means a NaN or +inf among them: look again at which
  uint32_t mine = any ? ord_of(big) : 0u;
  if (a.top > 0 && s.z != s.z) for_elements<BF16>(row, v0, v1, end_elem, [&](float x, int64_t) { mine = max(mine, ord_of(x)); });
  s = join_warp(s);
  if (lane == 0) stats[warp] = s;
  // the token's logit, ahead of its use
  float given = __int_as_float(0x7fc00000);              // no such token
  if (rank == 0 && tid == 0 && a.logprob != nullptr) {
    const int64_t tok = a.tokens[m];
    if (tok >= 0 && tok < a.V) given = row.at(tok);
  }
  const int live = static_cast<int>(v1 - v0 < kThreads ? v1 - v0 : kThreads), full = live / 32;
  const bool part = live % 32 >= 16 && live % 32 >= (a.top + full) / (full + 1);
  const int used = part ? full + 1 : full;             // 0: every element is a candidate, some hundred at most
  if (a.top > 0) {
    uint32_t left = mine, kth = 0;
    for (int j = 0; used > 0 && j < (a.top + used - 1) / used; ++j) {
      kth = __reduce_max_sync(0xffffffffu, left);
      const uint32_t who = __ballot_sync(0xffffffffu, left == kth);
      if (lane == __ffs(who) - 1) left = 0;
    }
    if (lane == 0) floor_of[warp] = kth;
  }
  if (tid == 0) found = 0;
  if (tid < kMaxTop) best[tid] = 0;
  __syncthreads();
  if (a.top > 0) {
    uint32_t floor = used > 0 ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) floor = min(floor, w < used ? floor_of[w] : floor);
    // A warp goes through its lanes that reach the floor, kSources at a time: the
    // 32 lanes load one's elements together.
    constexpr int kSources = 4;
    const float least = value_of(static_cast<uint64_t>(floor) << 32);
    auto offer = [&](float x, int64_t i) {
      if (x < least) return;                           // not a NaN
      const uint64_t key = argmax_key(x, static_cast<uint32_t>(i));
      if (static_cast<uint32_t>(key >> 32) < floor) return;
      const int at = atomicAdd(&found, 1);
      if (at < kCand) cand[at] = key;
    };
    uint32_t reach = __ballot_sync(0xffffffffu, any && mine >= floor);
    if (any && mine >= floor && end_elem >= 0) offer(row.at(end_elem), end_elem);
    if (live < kThreads) {                             // a load each: by the lanes themselves (60 rows of 15456 bf16, top 32: 10 instead of 62 us)
      if (reach >> lane & 1 && tid < live) {
        const uint4 u = row.load(v0 + tid);
#pragma unroll
        for (int e = 0; e < VE; ++e) offer(Row<BF16>::pick(u, e), row.head + (v0 + tid) * VE + e);
      }
      reach = 0;
    }
#pragma unroll 1
    while (reach != 0) {
      uint32_t some = reach;
#pragma unroll
      for (int k = 0; k < kSources; ++k) reach &= reach - 1;
      some &= ~reach;
#pragma unroll 1
      for (int64_t l = lane; v0 + warp * 32 + (l - lane) * kThreads < v1; l += 32) {
        uint4 u[kSources];
        uint32_t rest = some;
#pragma unroll
        for (int k = 0; k < kSources; ++k) {
          const int64_t v = v0 + warp * 32 + __ffs(rest) - 1 + l * kThreads;
          if (rest != 0 && v < v1) u[k] = row.load(v);
          rest &= rest - 1;
        }
        rest = some;
#pragma unroll
        for (int k = 0; k < kSources; ++k) {
          const int64_t v = v0 + warp * 32 + __ffs(rest) - 1 + l * kThreads;
          if (rest != 0 && v < v1) {
#pragma unroll
            for (int e = 0; e < VE; ++e) offer(Row<BF16>::pick(u[k], e), row.head + v * VE + e);
          }
          rest &= rest - 1;
        }
      }
    }
    __syncthreads();
    const int n = found;
    if (n <= kCand) {
      for (int c = tid; c < n; c += kThreads) {
        const uint64_t key = cand[c];
        int above = 0;
        for (int o = 0; o < n; ++o) above += cand[o] > key;
        if (above < a.top) best[above] = key;
      }
    } else {
      uint64_t prev = ~uint64_t(0);
      for (int k = 0; k < a.top; ++k) {
        uint64_t b = 0;
        for_elements<BF16>(row, v0, v1, end_elem, [&](float x, int64_t i) {
          const uint64_t key = argmax_key(x, static_cast<uint32_t>(i));
          if (key < prev) b = umax64(b, key);
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) b = umax64(b, __shfl_xor_sync(0xffffffffu, b, o));
        if (lane == 0) reduce[warp] = b;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) b = umax64(b, reduce[w]);
        if (tid == 0) best[k] = b;
        prev = b;
        __syncthreads();
        if (prev == 0) break;                          // fewer elements than asked for in this share
      }
    }
  }
  cluster.sync();
  if (rank == 0) {
    if (warp == 0) {
      constexpr int kEach = kWarps * kMaxCluster / 32;
      Stat t[kEach], all_t = {neg_inf(), 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int c = lane + 32 * k;
        t[k] = c < kWarps * C ? cluster.map_shared_rank(&stats[0], c / kWarps)[c % kWarps] : Stat{neg_inf(), 0.f, 0.f};
        all_t.m = fmaxf(all_t.m, t[k].m);
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        move_to(t[k], all_t.m);
        all_t.z += t[k].z;
        all_t.w += t[k].w;
      }
      all_t = join_warp(all_t);
      if (lane == 0) {
        const bool none = all_t.z == 0.f;                // every logit is -inf
        const float log_z = none ? neg_inf() : logf(all_t.z);
        const float lse = all_t.m + log_z;
        final_lse = lse;
        if (a.lse != nullptr) a.lse[m] = lse;
        if (a.entropy != nullptr) a.entropy[m] = none ? 0.f : log_z - all_t.w / all_t.z;
        if (a.logprob != nullptr) a.logprob[m] = none && given == given ? neg_inf() : given - lse;
      }
    } else {
      for (int e = tid - 32; e < a.top * C; e += kThreads - 32) {
        const int c = e / a.top;
        all[e] = cluster.map_shared_rank(&best[0], c)[e - c * a.top];
      }
    }
    __syncthreads();
    const int n = a.top * C;
    if (tid < n) {
      const uint64_t key = all[tid];
      int above = 0;
      for (int o = 0; o < n; ++o) above += all[o] > key;
      if (key != 0 && above < a.top) {
        const float lse = final_lse;
        a.top_idx[m * a.top + above] = argmax_index(key);
        a.top_lp[m * a.top + above] = lse == neg_inf() ? neg_inf() : value_of(key) - lse;
      }
    }
  }
  cluster.sync();                                      // peers keep their shared memory until rank 0 has read it
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsCall& c, const DeviceInfo& info, cudaStream_t s) {
  Args a;
  a.logits = static_cast<const uint8_t*>(c.logits);
  a.V = c.V;
  a.pitch = c.stride * (c.f32 ? 4 : 2);
  a.tokens = c.tokens;
  a.logprob = c.logprob;
  a.entropy = c.entropy;
  a.lse = c.lse;
  a.top_idx = c.top_idx;
  a.top_lp = c.top_lp;
  a.top = c.top;
  // As many CTAs a row as keep all rows' CTAs (two per SM) on the GPU at once (cold L2): 64 rows
  // of 151936 by 4 CTAs each 22, by 8 31, by 1 29 us; one row by 8 14, by 1 25.  The
  // last places take no whole cluster of 4 or 8: 38 rows by 8 19 us, by 4 14; 76 by 4 20, by 2 15.5.
  int cluster = kMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(c.M) * cluster > 2 * info.sms - (cluster > 2 ? 2 * cluster : 0)) cluster /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster), static_cast<unsigned>(c.M));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return c.f32 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<false>, a) : cudaLaunchKernelEx(&cfg, logprobs_kernel<true>, a);
}

}  // namespace q4nx
