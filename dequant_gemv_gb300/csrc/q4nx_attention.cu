// q4nx_attention.cu -- attention of a few query rows over the 4-bit cache.
//
//   out[r] = sum_j p[r][j] v[j] / sum_j p[r][j],   p[r][j] = exp(scale * q[r].k[j])
// over the positions j that row r sees (j <= its own position, and j > that
// minus the window where there is one); k = (ck - 8)*sk + mk and v likewise
// per group g of 32 channels.  One pass with a running reference per row.
//
// Keys enter as exact fp16 codes (a code's bits are the subnormal c*2^-24: one
// AND makes two), queries as fp16 scaled by a power of two per row (bf16 has
// 8 significant bits, so nothing is lost above 2^-39 of the row's largest), and
// the scales meet the products in binary32:
//   q.k   = sum_g sk_g * (q_g.ck_g - 8*Q_g) + mk_g * Q_g,  Q_g = sum of q over g
//   out_g = sum_j (p sv_g) (cv - 8) + sum_j p mv_g
// -8*Q_g is the matrix product's initial accumulator; mk_g*Q_g is a matrix
// product with Q_g as three bf16 parts (24 bits), sum_j p mv_g one with p as
// two (16 bits).  The values' codes are centred before their product (fp16
// 1024 + c, less 1032): sums over thousands of tokens stay near their result.
// p*sv is rounded to fp16 (2^-11 of itself; a power of two per row, which
// follows the largest p*sv seen, keeps it in range); bf16 values would cost
// 2^-9.  Codes in the high nibble of a byte enter as 16c: their q is divided
// by 16, and so are the sums of the values' upper 8 channels of 16.
//
// Tokens are the M of the products and query rows the N (8 per tile): a
// decode step has as few rows as query heads share a kv head, and padding
// them to an M of 16 would double the products.  S^T comes out with a lane's
// rows side by side; movmatrix turns p*sv into the B operand of the second
// product.
//
// Work: units (request, kv head, group of NT*8 query rows); their 16-token
// blocks form one sequence that the CTAs divide evenly, so ragged lengths need
// no plan.  A CTA has kWarps consumer warps, each taking every kWarps-th block
// of the CTA's range from a ring of block copies that a producer warp keeps
// full (lane = ring stage: each lane looks up its own pages and issues its own
// bulk copy).  Units that end inside a CTA's range leave finished; a unit
// split between CTAs leaves partial sums, and the CTA that posts last joins
// them in the order of the CTAs, so the result does not depend on timing.
#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

namespace q4nx {

namespace {

constexpr int kWarps = 7;                        // consumer warps; with the producer 8, so that 128 (two CTAs per SM) or 255 registers are left a thread
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kRefNone = -3.0e38f;             // reference of a row that has seen nothing
constexpr int kSnapBlocks = 16;                  // units up to this many blocks are not split
constexpr int kMinBlocks = 8;                    // fewer blocks than this are not worth a CTA

// A multiple of kWarps: one warp consumes all phases of a stage in order (a
// warp ahead of another by two phases would take an old phase's completion for its own).
__host__ __device__ constexpr int ring_stages(int D) { return kWarps * (D == 256 ? 2 : D == 128 ? 3 : 4); }
__host__ __device__ constexpr int row_pitch(int D) { return D + 4; }   // floats; rows 2i of a store fall on different banks
__host__ __device__ constexpr size_t attention_smem(int D, int NT) {
  return static_cast<size_t>(ring_stages(D)) * kv_block_bytes(D) +          // ring
         static_cast<size_t>(kWarps) * 8 * NT * row_pitch(D) * 4 +          // the warps' sums
         static_cast<size_t>(kWarps) * 8 * NT * 2 * 4 +                     // their references and totals
         ring_stages(D) * 16 + (kKvMaxBatch + 1) * 8 + 16;
}

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
  float* partial;           // [2*grid][RB][D + 2]
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
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

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

// How the blocks of all units are divided: position x of 0..total-1 is block
// x - unit_start of a unit; the units of request b begin at prefix[b].
struct Plan {
  const int64_t* prefix;    // shared memory, [batch + 1]
  int64_t total;
  int ctas;
  int batch;
};

struct Unit {
  int b, h;
  int64_t rg;               // group of RB query rows
  int64_t start, n;         // first position, number of blocks
  int64_t first_block;      // first 16-token block of the request that any row sees
  KvRequest rq;
};

__device__ __forceinline__ int64_t first_visible_block(const KvRequest& rq, int64_t window) {
  if (window <= 0) return 0;
  const int64_t f = rq.L - rq.T + 1 - window;
  return f > 0 ? f / kKvBlock : 0;
}
__device__ __forceinline__ int64_t unit_blocks(const KvRequest& rq, int64_t window) {
  const int64_t n = (rq.L + kKvBlock - 1) / kKvBlock - first_visible_block(rq, window);
  return n > 0 ? n : 1;     // an empty request's rows are written too
}

template <int RB>
__device__ Unit find_unit(const AttnArgs& a, const Plan& pl, int64_t x) {
  int lo = 0, hi = pl.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  Unit u;
  u.b = lo;
  u.rq = kv_request(a.kb, a.pool.page_blocks, lo);
  u.n = unit_blocks(u.rq, a.window);
  u.first_block = first_visible_block(u.rq, a.window);
  const int64_t groups = (u.rq.T * a.group + RB - 1) / RB;
  const int64_t k = (x - pl.prefix[lo]) / u.n;
  u.h = static_cast<int>(k / groups);
  u.rg = k - u.h * groups;
  u.start = pl.prefix[lo] + k * u.n;
  return u;
}

// First position of CTA c: an even share, moved to the end of the unit it
// falls into where that unit is too small to be split.
template <int RB>
__device__ int64_t bound(const AttnArgs& a, const Plan& pl, int c) {
  if (c >= pl.ctas) return pl.total;
  const int64_t q = pl.total / pl.ctas, rest = pl.total - q * pl.ctas;
  const int64_t x = q * c + (c < rest ? c : rest);
  if (x >= pl.total) return pl.total;
  const Unit u = find_unit<RB>(a, pl, x);
  return (u.n <= kSnapBlocks && x != u.start) ? u.start + u.n : x;
}
// The CTA whose even share holds position x.
__device__ __forceinline__ int share_of(const Plan& pl, int64_t x) {
  const int64_t q = pl.total / pl.ctas, rest = pl.total - q * pl.ctas;
  return static_cast<int>(x < (q + 1) * rest ? x / (q + 1) : rest + (x - (q + 1) * rest) / q);
}

// The running state of a warp over its blocks of one piece of a unit.  Pairs
// (float2) belong to the lane's query rows 2i and 2i + 1.
template <int D, int NT>
struct State {
  static constexpr int NG = D / 32;
  uint32_t qb[NT][NG][4];        // q as B operands: [group][k-step of 16: b0 b1], times 2^(14 - e) of its row
  float2 q8[NT][NG];             // -8 * Q_g, in the products' unit: 2^(-10 - e)
  uint32_t qs[NT][(NG + 3) / 4][2];   // Q_g of row lane/4 in three bf16 parts, g = 4*half + i
  float2 cr[NT];                 // softmax scale * log2(e) * 2^(10 + e)
  float o[NT][D / 16][4];        // [channels 16mt + lane/4 (+8, times 16)][rows 2i, 2i+1], times fs
  float corr[NT][4];             // sum of p*mid, group lane/4, rows 2i, 2i+1 (then two unused)
  float2 ref[NT], l[NT];         // reference of p = 2^(logit - ref), sum of p
  float2 fs[NT];                 // the power of two on p * value scale
};

template <int D, int NT>
__device__ __forceinline__ void load_q(const AttnArgs& a, const Unit& u, State<D, NT>& st) {
  constexpr int NG = D / 32;
  const int lane = threadIdx.x & 31, i = lane & 3, n = lane >> 2;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t r = u.rg * (8 * NT) + 8 * t + n;
    const int64_t tq = r / a.group;
    const bool have = tq < u.rq.T;
    const uint16_t* src = a.q + (u.rq.q0 + tq) * a.q_stride + static_cast<int64_t>(u.h * a.group + static_cast<int>(r - tq * a.group)) * D;
    uint4 w[NG];
    float big = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      w[g] = make_uint4(0, 0, 0, 0);
      if (have) w[g] = __ldg(reinterpret_cast<const uint4*>(src + 32 * g + 8 * i));
      const uint32_t v[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) big = fmaxf(big, fmaxf(fabsf(bf_lo(v[j])), fabsf(bf_hi(v[j]))));
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;      // |q| < 2^(e + 1)
    e = e < -100 ? -100 : e > 116 ? 116 : e;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
    const float c = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 10 + e) << 23);
    st.cr[t] = make_float2(__shfl_sync(0xffffffffu, c, 8 * i), __shfl_sync(0xffffffffu, c, 8 * i + 4));
    float sum[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t v[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = bf_lo(v[j]) * up, y = bf_hi(v[j]) * up;
        s += x + y;
        const float f = j & 1 ? 0.0625f : 1.f;                       // those codes come as 16c
        st.qb[t][g][j] = pack_f16x2(x * f, y * f);
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s *= 0x1p-24f;
      sum[g] = s;
      st.q8[t][g] = make_float2(-8.f * __shfl_sync(0xffffffffu, s, 8 * i), -8.f * __shfl_sync(0xffffffffu, s, 8 * i + 4));
    }
#pragma unroll
    for (int hf = 0; hf < (NG + 3) / 4; ++hf) {
      float s = 0.f;                                        // lanes without a group of their own add nothing
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (g == 4 * hf + i) s = sum[g];
      const float hi = __bfloat162float(__float2bfloat16_rn(s));
      const float mid = __bfloat162float(__float2bfloat16_rn(s - hi));
      st.qs[t][hf][0] = pack_bf16x2(hi, mid);
      st.qs[t][hf][1] = pack_bf16x2((s - hi) - mid, 0.f);
    }
  }
}

template <int D, int NT>
__device__ __forceinline__ void reset(State<D, NT>& st) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int m = 0; m < D / 16; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][m][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) st.corr[t][e] = 0.f;
    st.ref[t] = both(kRefNone);
    st.l[t] = both(0.f);
    st.fs[t] = both(0x1p100f);
  }
}

// A row's new reference: y0, y1 its logits at this lane's two tokens, m0, m1
// those tokens' largest value scales.  Returns the factor on the row's O; *f is that
// on its sums of p.
__device__ __forceinline__ float move_reference(float y0, float y1, float m0, float m1, float& ref, float& fs, float* f) {
  float m = fmaxf(y0, y1);
#pragma unroll
  for (int x = 16; x > 2; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  m = fmaxf(m, ref);
  float tm = fmaxf(ex2(y0 - m) * m0, ex2(y1 - m) * m1);
#pragma unroll
  for (int x = 16; x > 2; x >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, x));
  *f = ex2(ref - m);
  const float back = inv_pow2(fs);
  tm = fmaxf(tm, *f * (512.f * back));                       // the largest p * scale so far
  int e = static_cast<int>(__float_as_uint(tm) >> 23) - 127;
  e = e < -91 ? -91 : e;
  const float now = __uint_as_float(static_cast<uint32_t>(127 + 9 - e) << 23);
  const float of = (*f * now) * back;
  ref = m;
  fs = now;
  return of;
}

// One block of 16 tokens (shared-memory address `blk`).  MASK: some row does
// not see some token; `seen` then has bit 4t + e set where row e&1 of tile t sees
// token lane/4 + 8*(e>>1).
template <int D, int NT, bool MASK>
__device__ __forceinline__ void block_step(State<D, NT>& st, uint32_t blk, uint32_t seen) {
  constexpr int NG = D / 32, NH = (NG + 3) / 4, NW = NG < 4 ? NG : 4;
  const int lane = threadIdx.x & 31, i = lane & 3, tk = lane >> 2;
  const float none = -__int_as_float(0x7f800000);
  float s[NT][4];
  // mid * Q
#pragma unroll
  for (int hf = 0; hf < NH; ++hf) {
    const int g = NG < 4 ? (i & (NG - 1)) : 4 * hf + i;
    const uint32_t z0 = lds_u16(blk + 17 * D + (tk * NG + g) * 2) * 0x10001u;
    const uint32_t z1 = lds_u16(blk + 17 * D + ((tk + 8) * NG + g) * 2) * 0x10001u;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (hf == 0) mma<false>(s[t], z0, z1, z0, z1, st.qs[t][hf][0], st.qs[t][hf][1], 0.f, 0.f, 0.f, 0.f);
      else mma_add<false>(s[t], z0, z1, z0, z1, st.qs[t][hf][0], st.qs[t][hf][1]);
    }
  }
#pragma unroll
  for (int hf = 0; hf < NH; ++hf) {
    uint32_t w0[NW], w1[NW];                                     // the codes of tokens tk and tk + 8
    lds_words<NW>(w0, blk + hf * 1024 + lane * (4 * NW));
    lds_words<NW>(w1, blk + hf * 1024 + (lane + 32) * (4 * NW));
    uint32_t s0[NW / 2], s1[NW / 2];
    lds_words<NW / 2>(s0, blk + 16 * D + tk * (2 * NG) + 8 * hf);
    lds_words<NW / 2>(s1, blk + 16 * D + (tk + 8) * (2 * NG) + 8 * hf);
#pragma unroll
    for (int gw = 0; gw < NW; ++gw) {
      const int g = 4 * hf + gw;
      const uint32_t x0 = w0[gw], x1 = w1[gw], y0 = x0 >> 8, y1 = x1 >> 8;
      constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;
      const float k0 = gw & 1 ? bf_hi(s0[gw >> 1]) : bf_lo(s0[gw >> 1]);
      const float k1 = gw & 1 ? bf_hi(s1[gw >> 1]) : bf_lo(s1[gw >> 1]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float acc[4];
        mma<true>(acc, x0 & kLo, x1 & kLo, x0 & kHi, x1 & kHi, st.qb[t][g][0], st.qb[t][g][1], st.q8[t][g].x, st.q8[t][g].y,
                  st.q8[t][g].x, st.q8[t][g].y);
        mma_add<true>(acc, y0 & kLo, y1 & kLo, y0 & kHi, y1 & kHi, st.qb[t][g][2], st.qb[t][g][3]);
        const float2 a = ffma2(both(k0), make_float2(acc[0], acc[1]), make_float2(s[t][0], s[t][1]));
        const float2 b = ffma2(both(k1), make_float2(acc[2], acc[3]), make_float2(s[t][2], s[t][3]));
        s[t][0] = a.x, s[t][1] = a.y, s[t][2] = b.x, s[t][3] = b.y;
      }
    }
  }
  // the value scales of tokens tk, tk + 8, and the largest of each
  uint32_t v0[NG / 2], v1[NG / 2];
  if constexpr (NG == 8) {
    lds_words<4>(v0, blk + 18 * D + tk * 16);
    lds_words<4>(v1, blk + 18 * D + (tk + 8) * 16);
  } else {
    lds_words<NG / 2>(v0, blk + 18 * D + tk * (2 * NG));
    lds_words<NG / 2>(v1, blk + 18 * D + (tk + 8) * (2 * NG));
  }
  float m0 = 0x1p-100f, m1 = 0x1p-100f;                          // not 0: a p without bound has to be seen
#pragma unroll
  for (int e = 0; e < NG / 2; ++e) {
    m0 = fmaxf(m0, fmaxf(bf_lo(v0[e]), bf_hi(v0[e])));
    m1 = fmaxf(m1, fmaxf(bf_lo(v1[e]), bf_hi(v1[e])));
  }
  // logits of tile t relative to `ref`, -inf where not seen
  auto logits = [&](int t, float2 ref, float2& y0, float2& y1) {
    y0 = ffma2(make_float2(s[t][0], s[t][1]), st.cr[t], ref);
    y1 = ffma2(make_float2(s[t][2], s[t][3]), st.cr[t], ref);
    if constexpr (MASK) {
      const uint32_t h = seen >> (4 * t);
      y0 = make_float2(h & 1 ? y0.x : none, h & 2 ? y0.y : none);
      y1 = make_float2(h & 4 ? y1.x : none, h & 8 ? y1.y : none);
    }
  };
  float2 p0[NT], p1[NT], f0[NT], f1[NT];                         // p at tokens tk, tk + 8; times fs
  auto weights = [&](int t) {
    float2 y0, y1;
    logits(t, make_float2(-st.ref[t].x, -st.ref[t].y), y0, y1);
    p0[t] = ex2(y0);
    p1[t] = ex2(y1);
    f0[t] = mul2(p0[t], st.fs[t]);
    f1[t] = mul2(p1[t], st.fs[t]);
  };
  float top = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    weights(t);
    top = fmaxf(top, fmaxf(fmaxf(f0[t].x, f0[t].y) * m0, fmaxf(f1[t].x, f1[t].y) * m1));
  }
  // The reference and the power of two move only when p * scale outgrows its
  // place (below 2^10 when it was set, 2^13 is let pass), so that most blocks
  // rescale nothing; a first block's p is infinite and moves them.
  if (__any_sync(0xffffffffu, top > 8192.f)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float2 y0, y1, f, of;
      logits(t, both(0.f), y0, y1);
      of.x = move_reference(y0.x, y1.x, m0, m1, st.ref[t].x, st.fs[t].x, &f.x);
      of.y = move_reference(y0.y, y1.y, m0, m1, st.ref[t].y, st.fs[t].y, &f.y);
      st.l[t] = mul2(st.l[t], f);
      st.corr[t][0] *= f.x;
      st.corr[t][1] *= f.y;
#pragma unroll
      for (int m = 0; m < D / 16; ++m) {
        st.o[t][m][0] *= of.x;
        st.o[t][m][1] *= of.y;
        st.o[t][m][2] *= of.x;
        st.o[t][m][3] *= of.y;
      }
      weights(t);
    }
  }
  // sum of p * mid: mids [group][token] as A, p in two bf16 parts as B
  {
    const int g = tk & (NG - 1);
    uint32_t z[2];
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(z[0]) : "r"(blk + 19 * D + g * 32 + 4 * i));
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(z[1]) : "r"(blk + 19 * D + g * 32 + 4 * i + 16));
    if constexpr (MASK) {
      // unseen tokens may hold anything, and 0 times it has to be 0; a NaN that a
      // row does see reaches it through the scale, which is NaN with the mid
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if ((z[e] & 0x7F80u) == 0x7F80u) z[e] &= 0xFFFF0000u;
        if ((z[e] & 0x7F800000u) == 0x7F800000u) z[e] &= 0xFFFFu;
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      st.l[t] = fadd2(st.l[t], fadd2(p0[t], p1[t]));
      const uint32_t h0 = pack_bf16x2(p0[t].x, p0[t].y), h1 = pack_bf16x2(p1[t].x, p1[t].y);
      const uint32_t r0 = pack_bf16x2(p0[t].x - bf_lo(h0), p0[t].y - bf_hi(h0));
      const uint32_t r1 = pack_bf16x2(p1[t].x - bf_lo(h1), p1[t].y - bf_hi(h1));
      mma_add<false>(st.corr[t], z[0], 0u, z[1], 0u, movmatrix(h0), movmatrix(h1));
      mma_add<false>(st.corr[t], z[0], 0u, z[1], 0u, movmatrix(r0), movmatrix(r1));
    }
  }
  // values: group g is the channel tiles 2g, 2g + 1
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    uint32_t w[4];
    lds_words<4>(w, blk + 8 * D + (q * 32 + lane) * 16);
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
      const int g = 2 * q + gg;
      const float u0 = g & 1 ? bf_hi(v0[g >> 1]) : bf_lo(v0[g >> 1]);
      const float u1 = g & 1 ? bf_hi(v1[g >> 1]) : bf_lo(v1[g >> 1]);
      uint32_t b[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float2 x0 = mul2(f0[t], both(u0)), x1 = mul2(f1[t], both(u1));
        if constexpr (MASK) {                                    // an unseen token's scale may be anything
          const uint32_t h = seen >> (4 * t);
          x0 = make_float2(h & 1 ? x0.x : 0.f, h & 2 ? x0.y : 0.f);
          x1 = make_float2(h & 4 ? x1.x : 0.f, h & 8 ? x1.y : 0.f);
        }
        b[t][0] = movmatrix(pack_f16x2(x0.x, x0.y));
        b[t][1] = movmatrix(pack_f16x2(x1.x, x1.y));
      }
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        // fp16 1024 + c less 1032, and 1024 + 16c less 1152
        const uint32_t x = w[2 * gg + mm], y = x >> 8;
        const uint32_t c0 = hadd2(lop3_and_or(x, 0x000F000Fu, 0x64006400u), 0xE408E408u);
        const uint32_t c1 = hadd2(lop3_and_or(x, 0x00F000F0u, 0x64006400u), 0xE480E480u);
        const uint32_t c2 = hadd2(lop3_and_or(y, 0x000F000Fu, 0x64006400u), 0xE408E408u);
        const uint32_t c3 = hadd2(lop3_and_or(y, 0x00F000F0u, 0x64006400u), 0xE480E480u);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_add<true>(st.o[t][2 * g + mm], c0, c1, c2, c3, b[t][0], b[t][1]);
      }
    }
  }
}

template <int D, int NT, typename Out>
__global__ void __launch_bounds__(kThreads, D == 256 || NT > 1 ? 1 : 2) attention_kernel(const AttnArgs a) {
  constexpr int RB = 8 * NT, S = ring_stages(D), BB = kv_block_bytes(D), NG = D / 32;
  static_assert(S % kWarps == 0 && S <= 32);
  extern __shared__ __align__(128) uint8_t smem[];
  float* sum = reinterpret_cast<float*>(smem + S * BB);                    // [warp][RB][row_pitch]
  float* ml = sum + kWarps * RB * row_pitch(D);                            // [warp][RB][2]
  uint64_t* full = reinterpret_cast<uint64_t*>(ml + kWarps * RB * 2);
  uint64_t* empty = full + S;
  int64_t* prefix = reinterpret_cast<int64_t*>(empty + S);
  int* flag = reinterpret_cast<int*>(prefix + kKvMaxBatch + 1);            // [0] joins, [1] a wait gave up
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the requests' blocks and their prefix sums
  const int B = a.kb.batch;
  for (int b = tid; b < B; b += kThreads) {
    const KvRequest rq = kv_request(a.kb, a.pool.page_blocks, b);
    if (!rq.ok && blockIdx.x == 0) atomicOr(a.err, kErrIndex);
    prefix[b + 1] = rq.T > 0 ? (rq.T * a.group + RB - 1) / RB * a.pool.kv_heads * unit_blocks(rq, a.window) : 0;
  }
  if (tid == 0) {
    prefix[0] = 0;
    flag[1] = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (warp == 0) {
    int64_t run = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int64_t v = b0 + lane < B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      v += run;
      if (b0 + lane < B) prefix[b0 + lane + 1] = v;
      run = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  Plan pl;
  pl.prefix = prefix;
  pl.total = prefix[B];
  pl.batch = B;
  const int64_t want = pl.total / kMinBlocks;
  pl.ctas = want < 1 ? 1 : want < gridDim.x ? static_cast<int>(want) : gridDim.x;
  if (pl.total == 0 || blockIdx.x >= pl.ctas) return;
  const int64_t begin = bound<RB>(a, pl, blockIdx.x), end = bound<RB>(a, pl, blockIdx.x + 1);
  if (begin >= end) return;

  if (warp == kWarps) {
    // ---- producer: lane s fills stage s ----
    if (lane < S) {
      uint32_t phase = 1;
      bool ok = true;
      Unit u = {};
      for (int64_t x = begin + lane; x < end; x += S) {
        if (x >= u.start + u.n) u = find_unit<RB>(a, pl, x);
        const int64_t blk = u.first_block + (x - u.start);
        const uint8_t* src = blk * kKvBlock < u.rq.L ? kv_block_ptr(a.pool, a.kb, D, u.b, u.h, blk) : nullptr;
        if (src == nullptr && blk * kKvBlock < u.rq.L) atomicOr(a.err, kErrIndex);
        if (!mbar_wait_bounded(&empty[lane], phase)) {           // a fresh barrier passes a wait for phase 1
          atomicOr(a.err, kErrTimeout);
          ok = false;
          break;
        }
        if (src != nullptr) {
          mbar_arrive_expect_tx(&full[lane], BB);
          bulk_g2s(smem + lane * BB, src, BB, &full[lane]);
        } else {
          mbar_arrive_expect_tx(&full[lane], 0);
        }
        phase ^= 1;
      }
      // the copy that nobody took (a wait gave up) lands before the CTA leaves
      if (!ok) mbar_wait_bounded(&full[lane], phase);
    }
    return;
  }

  // ---- consumers ----
  State<D, NT> st;
  const int i = lane & 3, tk = lane >> 2;
  const uint32_t ring = smem_u32(smem);
  for (int64_t ps = begin; ps < end;) {
    const Unit u = find_unit<RB>(a, pl, ps);
    const int64_t pe = u.start + u.n < end ? u.start + u.n : end;
    load_q<D, NT>(a, u, st);
    reset<D, NT>(st);
    const int64_t base = u.rq.L - u.rq.T;
    const int64_t row0 = u.rg * RB;
    const int64_t rows = u.rq.T * a.group - row0 < RB ? u.rq.T * a.group - row0 : RB;
    // blocks that every row sees whole: first_full <= block < end_full
    const int64_t pos_first = base + row0 / a.group, pos_last = base + (row0 + rows - 1) / a.group;
    const int64_t hidden = a.window > 0 ? pos_last - a.window : -1;          // the last position that some row does not see
    const int first_full = hidden < 0 ? 0 : static_cast<int>(hidden / kKvBlock + 1);
    const int end_full = pos_first < 0 ? 0 : static_cast<int>((pos_first + 1) / kKvBlock);
    // positions that this lane's rows see: lo < position <= hi (none for rows beyond the last)
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t r = row0 + 8 * t + 2 * i + e;
        const int64_t pos = base + r / a.group;
        hi[t][e] = static_cast<int>(pos < u.rq.L ? pos : u.rq.L - 1);
        lo[t][e] = static_cast<int>(a.window > 0 && pos - a.window > -1 ? pos - a.window : -1);
      }
    const int skip = static_cast<int>((ps - begin) % kWarps);
    uint32_t k = static_cast<uint32_t>(ps - begin) + (warp >= skip ? warp - skip : warp - skip + kWarps);
    const uint32_t k_end = static_cast<uint32_t>(pe - begin);
    const int blk0 = static_cast<int>(u.first_block + (ps - u.start)) - static_cast<int>(ps - begin);
    for (; k < k_end; k += kWarps) {
      const uint32_t round = k / S, stage = k - round * S;
      if (!mbar_wait_bounded(&full[stage], round & 1)) {
        flag[1] = 1;
        atomicOr(a.err, kErrTimeout);
        break;
      }
      const int blk = blk0 + static_cast<int>(k);
      const uint32_t addr = ring + stage * BB;
      if (blk >= first_full && blk < end_full) {
        block_step<D, NT, false>(st, addr, 0);
      } else {
        uint32_t seen = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = blk * kKvBlock + tk + 8 * (e >> 1);
            if (tok <= hi[t][e & 1] && tok > lo[t][e & 1]) seen |= 1u << (4 * t + e);
          }
        block_step<D, NT, true>(st, addr, seen);
      }
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[stage])) : "memory");
    }
    // this warp's sums, in the values' own units
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float2 back = make_float2(inv_pow2(st.fs[t].x), inv_pow2(st.fs[t].y));
#pragma unroll
      for (int o = 16; o > 2; o >>= 1) {
        st.l[t].x += __shfl_xor_sync(0xffffffffu, st.l[t].x, o);
        st.l[t].y += __shfl_xor_sync(0xffffffffu, st.l[t].y, o);
      }
      float* row = sum + (warp * RB + 8 * t + 2 * i) * row_pitch(D);
      float* next = row + row_pitch(D);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float z0 = __shfl_sync(0xffffffffu, st.corr[t][0], 4 * g + i), z1 = __shfl_sync(0xffffffffu, st.corr[t][1], 4 * g + i);
#pragma unroll
        for (int m = 2 * g; m < 2 * g + 2; ++m) {
          row[16 * m + tk] = fmaf(st.o[t][m][0], back.x, z0);
          next[16 * m + tk] = fmaf(st.o[t][m][1], back.y, z1);
          row[16 * m + tk + 8] = fmaf(st.o[t][m][2], 0.0625f * back.x, z0);
          next[16 * m + tk + 8] = fmaf(st.o[t][m][3], 0.0625f * back.y, z1);
        }
      }
      if (tk == 0) {
        float* at = ml + (warp * RB + 8 * t + 2 * i) * 2;
        at[0] = st.ref[t].x;
        at[1] = st.l[t].x;
        at[2] = st.ref[t].y;
        at[3] = st.l[t].y;
      }
    }
    bar_consumers();
    const bool whole = ps == u.start && pe == u.start + u.n;
    const int slot = 2 * blockIdx.x + (ps == begin ? 0 : 1);
    float* part = a.partial + static_cast<int64_t>(slot) * RB * (D + 2);
    for (int idx = tid; idx < static_cast<int>(rows) * D; idx += kWarps * 32) {
      const int r = idx / D, d = idx - r * D;
      float m = ml[r * 2];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, ml[(w * RB + r) * 2]);
      float o = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(ml[(w * RB + r) * 2] - m);
        o = fmaf(f, sum[(w * RB + r) * row_pitch(D) + d], o);
        l = fmaf(f, ml[(w * RB + r) * 2 + 1], l);
      }
      if (whole) {
        const int64_t rr = row0 + r, tq = rr / a.group;
        const int64_t at = (u.rq.q0 + tq) * a.heads + u.h * a.group + (rr - tq * a.group);
        const float y = l == 0.f ? 0.f : o / l;
        if constexpr (sizeof(Out) == 4) static_cast<float*>(a.out)[at * D + d] = y;
        else static_cast<uint16_t*>(a.out)[at * D + d] = f32_to_bf16_bits(y);
        if (d == 0 && a.lse != nullptr) a.lse[at] = l == 0.f ? -__int_as_float(0x7f800000) : (m + lg2(l)) * 0.693147180559945f;
      } else {
        __stcg(part + r * D + d, o);
        if (d == 0) {
          __stcg(part + RB * D + 2 * r, m);
          __stcg(part + RB * D + 2 * r + 1, l);
        }
      }
    }
    if (!whole) {
      // the CTAs that hold a piece of this unit; the last one to post joins them
      const int c0 = share_of(pl, u.start), c1 = share_of(pl, u.start + u.n - 1);
      __threadfence();
      bar_consumers();
      if (tid == 0) {
        const uint32_t before = atomicAdd(a.counters + c0, 1u);
        const bool last = before == static_cast<uint32_t>(c1 - c0);
        if (last) a.counters[c0] = 0;
        flag[0] = last;
      }
      bar_consumers();
      if (flag[0]) {
        __threadfence();
        // CTA c0's piece is its first one only where its range begins with the unit
        const int first = 2 * c0 + (bound<RB>(a, pl, c0) == u.start ? 0 : 1);
        const int64_t pitch = static_cast<int64_t>(RB) * (D + 2);
        const float* p0 = a.partial + first * pitch;
        for (int idx = tid; idx < static_cast<int>(rows) * D; idx += kWarps * 32) {
          const int r = idx / D, d = idx - r * D;
          float m = __ldcg(p0 + RB * D + 2 * r);
          for (int c = c0 + 1; c <= c1; ++c) m = fmaxf(m, __ldcg(a.partial + 2 * c * pitch + RB * D + 2 * r));
          float f = ex2(__ldcg(p0 + RB * D + 2 * r) - m);
          float o = f * __ldcg(p0 + r * D + d), l = f * __ldcg(p0 + RB * D + 2 * r + 1);
#pragma unroll 4
          for (int c = c0 + 1; c <= c1; ++c) {
            const float* p = a.partial + 2 * c * pitch;
            f = ex2(__ldcg(p + RB * D + 2 * r) - m);
            o = fmaf(f, __ldcg(p + r * D + d), o);
            l = fmaf(f, __ldcg(p + RB * D + 2 * r + 1), l);
          }
          const int64_t rr = row0 + r, tq = rr / a.group;
          const int64_t at = (u.rq.q0 + tq) * a.heads + u.h * a.group + (rr - tq * a.group);
          const float y = l == 0.f ? 0.f : o / l;
          if constexpr (sizeof(Out) == 4) static_cast<float*>(a.out)[at * D + d] = y;
          else static_cast<uint16_t*>(a.out)[at * D + d] = f32_to_bf16_bits(y);
          if (d == 0 && a.lse != nullptr) a.lse[at] = l == 0.f ? -__int_as_float(0x7f800000) : (m + lg2(l)) * 0.693147180559945f;
        }
      }
    }
    bar_consumers();                                             // the sums are read out
    if (flag[1]) break;
    ps = pe;
  }
}

template <int D, int NT, typename Out>
cudaError_t launch_variant(const AttnArgs& a, int grid, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(attention_kernel<D, NT, Out>);
  cudaError_t e = set_max_dynamic_smem(f);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = attention_smem(D, NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_kernel<D, NT, Out>, a);
}

}  // namespace

uint64_t attention_workspace_bytes(int D) {
  return 16 + kKvMaxCtas * 4 + static_cast<uint64_t>(2 * kKvMaxCtas) * 16 * (D + 2) * 4;
}

cudaError_t launch_attention(int D, const KvPool& pool, const KvBatch& kb, const void* q, int64_t q_stride, int heads,
                             float scale, int64_t window, void* out, int out_f32, float* lse, void* workspace,
                             const DeviceInfo& info, cudaStream_t s) {
  AttnArgs a;
  a.pool = pool;
  a.kb = kb;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.heads = heads;
  a.group = heads / pool.kv_heads;
  a.scale_log2 = scale * 1.44269504088896f;
  a.window = window;
  a.out = out;
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + 16);
  a.partial = reinterpret_cast<float*>(ws + 16 + kKvMaxCtas * 4);
  // rows per request on average decide the tile: one of 8 rows, or two that share each block's decoding
  const int64_t rows = kb.tokens * a.group;
  const bool two = rows > static_cast<int64_t>(8) * kb.batch;
  const int per_sm = D == 256 || two ? 1 : 2;
  const int grid = info.sms * per_sm < kKvMaxCtas ? info.sms * per_sm : kKvMaxCtas;
#define Q4NX_ATTN(DD)                                                                                             \
  case DD:                                                                                                        \
    return two ? (out_f32 ? launch_variant<DD, 2, float>(a, grid, s) : launch_variant<DD, 2, uint16_t>(a, grid, s)) \
               : (out_f32 ? launch_variant<DD, 1, float>(a, grid, s) : launch_variant<DD, 1, uint16_t>(a, grid, s));
  switch (D) {
    Q4NX_ATTN(64)
    Q4NX_ATTN(128)
    Q4NX_ATTN(256)
    default: return cudaErrorInvalidValue;
  }
#undef Q4NX_ATTN
}

}  // namespace q4nx
