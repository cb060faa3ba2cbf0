// q4nx_attention_rows.cuh -- attention of a few query rows over the 4-bit cache.
//
//   out[r] = sum_j p[r][j] v[j] / sum_j p[r][j],   p[r][j] = exp(scale * q[r].k[j])
// over the positions j that row r sees (j <= its own position, and j > that
// minus the window where there is one); k = (ck - 8)*sk + mk and v likewise
// per group g of 32 channels.  One pass with a running reference per row.
//
// Keys enter as exact fp16 codes (a code's bits are the subnormal c*2^-24: one
// AND makes two), queries as fp16 scaled by a power of two per row (bf16 has
// 8 significant bits, so nothing is lost above 2^-27 of the row's largest, and 2^-35
// of it at most below; rows of 2^117 and more would overflow), and the scales meet the
// products in binary32:
//   q.k   = sum_g sk_g * (q_g.ck_g) + sk_g * (-8*Q_g) + mk_g * Q_g,  Q_g = sum of q over g
//   out_g = sum_j (p sv_g) (cv - 8) + sum_j p mv_g
// The two terms with Q_g are matrix products with it as three bf16 parts (24
// bits; as the products' initial accumulator -8*Q_g cost four moves each),
// sum_j p mv_g is one with p as two (16 bits).  The values' codes are centred before their product (fp16
// 1024 + c, less 1032): sums over thousands of tokens stay near their result.
// p*sv is rounded to fp16 (2^-11 of itself; a power of two per row, which
// keeps the largest p*sv seen between 2^9 and 2^13, so that products 2^-23 of it and
// less are subnormal, rounded by 2^-34 of it); bf16 values would cost 2^-9.  Codes in
// the high nibble of a byte enter as 16c: their q is divided by 16, and so are the sums
// of the values' upper 8 channels of 16.
//
// Tokens are the M of the products and query rows the N (8 per tile): a
// decode step has as few rows as query heads share a kv head, and padding
// them to an M of 16 would double the products.  S^T comes out with a lane's
// rows side by side; movmatrix turns p*sv into the B operand of the second
// product.
//
// Work: units (request, kv head, group of NT*8 query rows); their 32-token
// steps form one sequence of positions, divided between the CTAs so that ragged
// lengths need no plan (a unit counts kUnitCost steps more than it has, for
// its beginning and end), and a CTA's range evenly between its warps.  A warp
// goes through its positions by itself and keeps copies of its next steps in
// flight in a ring of its own: its lanes look up the pages of 32 steps at a
// time, and lane 0 sends the next copy as soon as a stage is read out.  A unit
// that ends inside a warp's range is written from its registers; what the
// ranges cut is joined once, at the CTA's end, in shared memory, and units cut
// between CTAs by the CTA that posts last, in the order of the CTAs, so that the
// result does not depend on timing.  (With all warps of a CTA on one unit at
// a time every unit cost the CTA 4 us of waiting and joining: 71 us instead
// of 58 for 48 requests of 600 to 6000 tokens, 8 kv heads.)
//
// Bound: these 209 MB take 56.3 us, 3.7 TB/s or 55% of a copy's rate.  A block of 16
// tokens x 128 channels of keys and values costs 395 instructions of a warp; the
// schedulers issue 53% of the time, the rest goes to fixed latencies within a
// warp (four warps a scheduler, for the registers' sake) and to the 8 to 10 us in
// which a CTA makes its plan, waits for its first copies and joins its parts.
#pragma once

#include "q4nx_attention.cuh"

namespace q4nx {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// 16-token blocks of one step (a ring stage), and stages of a warp's ring
__host__ __device__ constexpr int step_blocks(int D) { return D == 256 ? 1 : 2; }
__host__ __device__ constexpr int ring_stages(int D) { return D == 128 ? 2 : 4; }
__host__ __device__ constexpr int stage_bytes(int D) { return step_blocks(D) * kv_block_bytes(D); }

// The piece of a unit that a warp works on: what it has to know of it, in
// shared memory (in registers it would push the running sums out).
template <int RB>
struct Piece {
  int64_t q0, row0, T;      // first token of the request, first query row of the unit, tokens of the request
  int64_t start, n, cost;   // the unit's first position, its steps, the costs before it
  int h, rows;              // kv head, query rows
  int first_full, end_full; // steps of the request that every row sees whole
  int step0;                // the request's step at the warp's first position, as if the unit went back there
  int end;                  // where the piece ends, in steps from the warp's first position
  bool whole;               // all of the unit
  bool split;               // its rows have another part, in another pass
  int lo[RB], hi[RB];       // a row sees positions lo < p <= hi
};

// What is left to know of a unit of which a warp has a part.
struct Cut {
  int64_t q0, row0, start, n, cost;
  int h, rows;
  bool split;
};

template <int D, int NT, int SEE>
struct Smem {
  static constexpr int RB = 8 * NT, S = ring_stages(D);
  alignas(128) uint8_t ring[kWarps][S][stage_bytes(D)];
  uint64_t full[kWarps][S];
  alignas(16) const uint8_t* src[kWarps][32][step_blocks(D)];   // where the blocks of a warp's next 32 steps lie
  Piece<RB> piece[kWarps];
  // A warp's parts of cut units, entry 2*warp for the unit it began with, 2*warp
  // + 1 for the one it ended with (start -1: none): reference and total of each row
  Cut cut[2 * kWarps];
  float2 ml[2 * kWarps][RB];
  float2 total[2 * kWarps][RB];                       // those of the CTA's parts of the unit together
  int64_t prefix[kKvMaxBatch + 1], cost[kKvMaxBatch + 1];
  int longest[32];
  int64_t begin, end;
  int stopped, joins[2];
  int lower[SEE == kOwn ? kKvMaxBatch : 1];
};

// The running state of a warp over its blocks of one piece of a unit.  Pairs
// (float2) belong to the lane's query rows 2i and 2i + 1.
template <int D, int NT>
struct State {
  static constexpr int NG = D / 32;
  uint32_t qb[NT][NG][4];        // q as B operands: [group][k-step of 16: b0 b1], times 2^(14 - e) of its row
  // Q_g and -8 * Q_g of row lane/4 in three bf16 parts, g = 4*half + i, in the products' unit 2^(-10 - e)
  uint32_t qs[2][NT][(NG + 3) / 4][2];
  float2 cr[NT];                 // softmax scale * log2(e) * 2^(10 + e)
  float o[NT][D / 16][4];        // [channels 16mt + lane/4 (+8, times 16)][rows 2i, 2i+1], times fs
  float corr[NT][4];             // sum of p*mid, group lane/4, rows 2i, 2i+1 (then two unused)
  float2 ref[NT], l[NT];         // reference of p = 2^(logit - ref), sum of p
  float2 fs[NT];                 // the power of two on p * value scale
};

template <int D, int NT, class A>
__device__ __forceinline__ void load_q(const A& a, const Piece<8 * NT>& u, State<D, NT>& st) {
  constexpr int NG = D / 32;
  const int lane = threadIdx.x & 31, i = lane & 3, n = lane >> 2;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t r = u.row0 + 8 * t + n;
    const int64_t tq = quot(r, a.group);
    const bool have = tq < u.T;
    const uint16_t* src = a.q + (u.q0 + tq) * a.q_stride + static_cast<int64_t>(u.h * a.group + static_cast<int>(r - tq * a.group)) * D;
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
    }
#pragma unroll
    for (int hf = 0; hf < (NG + 3) / 4; ++hf) {
      float s = 0.f;                                        // lanes without a group of their own add nothing
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (g == 4 * hf + i) s = sum[g];
      const float hi = __bfloat162float(__float2bfloat16_rn(s));
      const float mid = __bfloat162float(__float2bfloat16_rn(s - hi));
      st.qs[0][t][hf][0] = pack_bf16x2(hi, mid);
      st.qs[0][t][hf][1] = pack_bf16x2((s - hi) - mid, 0.f);
      st.qs[1][t][hf][0] = pack_bf16x2(-8.f * hi, -8.f * mid);
      st.qs[1][t][hf][1] = pack_bf16x2(-8.f * ((s - hi) - mid), 0.f);
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

// A row's new reference: y(n) its logits at this lane's two tokens of block n,
// m0, m1 those tokens' largest value scales.  Returns the factor on the row's O;
// *f is that on its sums of p.
template <int NB, typename Y>
__device__ __forceinline__ float move_reference(Y y, const float (&m0)[NB], const float (&m1)[NB], float& ref, float& fs, float* f) {
  float m = ref;
#pragma unroll
  for (int n = 0; n < NB; ++n) m = fmaxf(m, fmaxf(y(n).x, y(n).y));
#pragma unroll
  for (int x = 16; x > 2; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float tm = 0.f;
#pragma unroll
  for (int n = 0; n < NB; ++n) tm = fmaxf(tm, fmaxf(ex2(y(n).x - m) * m0[n], ex2(y(n).y - m) * m1[n]));
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

// NB blocks of 16 tokens (shared-memory address `blk0`), taken together: two
// give the scheduler twice the independent work between the dependent stages
// (34.3 us for the loop over 131071 tokens; 35.6 one at a time).  Where `full` is
// not set some row does not see some token: bit 4t + e of seen[n] is set where
// row e&1 of tile t sees token lane/4 + 8*(e>>1) of block n, and clear_hidden has
// made the blocks' values finite.
template <int D, int NT, int NB>
__device__ __forceinline__ void block_step(State<D, NT>& st, uint32_t blk0, bool full, const uint32_t (&seen)[NB]) {
  constexpr int NG = D / 32, NH = (NG + 3) / 4, NW = NG < 4 ? NG : 4, BB = kv_block_bytes(D);
  const int lane = threadIdx.x & 31, i = lane & 3, tk = lane >> 2;
  const float none = -__int_as_float(0x7f800000);
  float s[NB][NT][4];
  uint32_t v0[NB][NG / 2], v1[NB][NG / 2];                       // value scales of tokens tk, tk + 8
  float m0[NB], m1[NB];                                          // the largest of each token
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const uint32_t blk = blk0 + n * BB;
    // mid * Q - 8 * scale * Q
#pragma unroll
    for (int hf = 0; hf < NH; ++hf) {
      const int g = NG < 4 ? (i & (NG - 1)) : 4 * hf + i;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t z0 = lds_u16(blk + (17 - k) * D + (tk * NG + g) * 2) * 0x10001u;
        const uint32_t z1 = lds_u16(blk + (17 - k) * D + ((tk + 8) * NG + g) * 2) * 0x10001u;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (hf == 0 && k == 0) mma<false>(s[n][t], z0, z1, z0, z1, st.qs[k][t][hf][0], st.qs[k][t][hf][1], 0.f, 0.f, 0.f, 0.f);
          else mma_add<false>(s[n][t], z0, z1, z0, z1, st.qs[k][t][hf][0], st.qs[k][t][hf][1]);
        }
      }
    }
#pragma unroll
    for (int hf = 0; hf < NH; ++hf) {
      uint32_t w0[NW], w1[NW];                                   // the codes of tokens tk and tk + 8
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
          mma<true>(acc, x0 & kLo, x1 & kLo, x0 & kHi, x1 & kHi, st.qb[t][g][0], st.qb[t][g][1], 0.f, 0.f, 0.f, 0.f);
          mma_add<true>(acc, y0 & kLo, y1 & kLo, y0 & kHi, y1 & kHi, st.qb[t][g][2], st.qb[t][g][3]);
          const float2 a = ffma2(both(k0), make_float2(acc[0], acc[1]), make_float2(s[n][t][0], s[n][t][1]));
          const float2 b = ffma2(both(k1), make_float2(acc[2], acc[3]), make_float2(s[n][t][2], s[n][t][3]));
          s[n][t][0] = a.x, s[n][t][1] = a.y, s[n][t][2] = b.x, s[n][t][3] = b.y;
        }
      }
    }
    if constexpr (NG == 8) {
      lds_words<4>(v0[n], blk + 18 * D + tk * 16);
      lds_words<4>(v1[n], blk + 18 * D + (tk + 8) * 16);
    } else {
      lds_words<NG / 2>(v0[n], blk + 18 * D + tk * (2 * NG));
      lds_words<NG / 2>(v1[n], blk + 18 * D + (tk + 8) * (2 * NG));
    }
    m0[n] = m1[n] = 0x1p-100f;                                   // not 0: a p without bound has to be seen
#pragma unroll
    for (int e = 0; e < NG / 2; ++e) {
      m0[n] = fmaxf(m0[n], fmaxf(bf_lo(v0[n][e]), bf_hi(v0[n][e])));
      m1[n] = fmaxf(m1[n], fmaxf(bf_lo(v1[n][e]), bf_hi(v1[n][e])));
    }
  }
  // logits of tile t relative to `ref`, -inf where not seen
  auto logits = [&](int n, int t, float2 ref, float2& y0, float2& y1) {
    y0 = ffma2(make_float2(s[n][t][0], s[n][t][1]), st.cr[t], ref);
    y1 = ffma2(make_float2(s[n][t][2], s[n][t][3]), st.cr[t], ref);
    if (!full) {
      const uint32_t h = seen[n] >> (4 * t);
      y0 = make_float2(h & 1 ? y0.x : none, h & 2 ? y0.y : none);
      y1 = make_float2(h & 4 ? y1.x : none, h & 8 ? y1.y : none);
    }
  };
  float2 p0[NB][NT], p1[NB][NT];                                 // p at tokens tk, tk + 8
  auto weights = [&](int t) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float2 y0, y1;
      logits(n, t, make_float2(-st.ref[t].x, -st.ref[t].y), y0, y1);
      p0[n][t] = ex2(y0);
      p1[n][t] = ex2(y1);
    }
  };
  float top = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    weights(t);
    float2 big = both(0.f);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      big.x = fmaxf(big.x, fmaxf(p0[n][t].x * m0[n], p1[n][t].x * m1[n]));
      big.y = fmaxf(big.y, fmaxf(p0[n][t].y * m0[n], p1[n][t].y * m1[n]));
    }
    top = fmaxf(top, fmaxf(big.x * st.fs[t].x, big.y * st.fs[t].y));
  }
  // The reference and the power of two move only when p * scale outgrows its
  // place (below 2^10 when it was set, 2^13 is let pass), so that most steps
  // rescale nothing; a first step's p is infinite and moves them.
  if (__any_sync(0xffffffffu, top > 8192.f)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float2 y0[NB], y1[NB], f, of;
#pragma unroll
      for (int n = 0; n < NB; ++n) logits(n, t, both(0.f), y0[n], y1[n]);
      of.x = move_reference<NB>([&](int n) { return make_float2(y0[n].x, y1[n].x); }, m0, m1, st.ref[t].x, st.fs[t].x, &f.x);
      of.y = move_reference<NB>([&](int n) { return make_float2(y0[n].y, y1[n].y); }, m0, m1, st.ref[t].y, st.fs[t].y, &f.y);
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
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const uint32_t blk = blk0 + n * BB;
    // sum of p * mid: mids [group][token] as A, p in two bf16 parts as B
    const int g0 = tk & (NG - 1);
    uint32_t z[2];
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(z[0]) : "r"(blk + 19 * D + g0 * 32 + 4 * i));
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(z[1]) : "r"(blk + 19 * D + g0 * 32 + 4 * i + 16));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float2 q0 = p0[n][t], q1 = p1[n][t];
      st.l[t] = fadd2(st.l[t], fadd2(q0, q1));
      const uint32_t h0 = pack_bf16x2(q0.x, q0.y), h1 = pack_bf16x2(q1.x, q1.y);
      const uint32_t r0 = pack_bf16x2(q0.x - bf_lo(h0), q0.y - bf_hi(h0));
      const uint32_t r1 = pack_bf16x2(q1.x - bf_lo(h1), q1.y - bf_hi(h1));
      mma_add<false>(st.corr[t], z[0], 0u, z[1], 0u, movmatrix(h0), movmatrix(h1));
      mma_add<false>(st.corr[t], z[0], 0u, z[1], 0u, movmatrix(r0), movmatrix(r1));
      p0[n][t] = mul2(q0, st.fs[t]);
      p1[n][t] = mul2(q1, st.fs[t]);
    }
    // values: group g is the channel tiles 2g, 2g + 1
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
      uint32_t w[4];
      lds_words<4>(w, blk + 8 * D + (q * 32 + lane) * 16);
#pragma unroll
      for (int gg = 0; gg < 2; ++gg) {
        const int g = 2 * q + gg;
        const float u0 = g & 1 ? bf_hi(v0[n][g >> 1]) : bf_lo(v0[n][g >> 1]);
        const float u1 = g & 1 ? bf_hi(v1[n][g >> 1]) : bf_lo(v1[n][g >> 1]);
        uint32_t b[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 x0 = mul2(p0[n][t], both(u0)), x1 = mul2(p1[n][t], both(u1));
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
}

// The rows that see the tokens of block `blk` (16 positions), as block_step wants them.
template <int NT>
__device__ __forceinline__ uint32_t seen_bits(const Piece<8 * NT>& u, int blk) {
  const int lane = threadIdx.x & 31, i = lane & 3, tk = lane >> 2;
  uint32_t seen = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 8 * t + 2 * i + (e & 1), tok = blk * kKvBlock + tk + 8 * (e >> 1);
      if (tok <= u.hi[r] && tok > u.lo[r]) seen |= 1u << (4 * t + e);
    }
  return seen;
}

// Makes 0 * value 0 in a block (address `at`, 16 positions from tok0) that some
// row does not see whole.  Tokens that no row sees may hold anything: their value
// scales and mids become 0.  A token that some rows see may be kept as NaN:
// it becomes 0 too, and the rows that see it get their NaN here, in that group
// alone (its logit, where the key is NaN, is masked row by row in any case).
template <int D, int NT>
__device__ __forceinline__ void clear_hidden(State<D, NT>& st, const Piece<8 * NT>& u, uint32_t at, int tok0, uint32_t seen) {
  constexpr int NG = D / 32;
  const int lane = threadIdx.x & 31, i = lane & 3, tk = lane >> 2;
  bool odd = false;                                              // a scale that is no number, on this lane's token
  if (lane < kKvBlock) {
    const bool hidden = tok0 + lane <= u.lo[0] || tok0 + lane > u.hi[u.rows - 1];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t s_at = at + 18 * D + (lane * NG + g) * 2, m_at = at + 19 * D + (g * kKvBlock + lane) * 2;
      if (hidden) {
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(s_at), "h"(static_cast<uint16_t>(0)) : "memory");
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(m_at), "h"(static_cast<uint16_t>(0)) : "memory");
      } else {
        odd |= (lds_u16(s_at) & 0x7F80u) == 0x7F80u;
      }
    }
  }
  if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
    for (int g = 0; g < NG; ++g) {
      bool bad[2];                                               // this lane's tokens tk, tk + 8
#pragma unroll
      for (int h = 0; h < 2; ++h) bad[h] = (lds_u16(at + 18 * D + ((tk + 8 * h) * NG + g) * 2) & 0x7F80u) == 0x7F80u;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool hit = (bad[0] && (seen >> (4 * t + e) & 1)) || (bad[1] && (seen >> (4 * t + e + 2) & 1));
          if (__ballot_sync(0xffffffffu, hit) & (0x11111111u << i))
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
              if ((m >> 1) == g) st.o[t][m][e] = st.o[t][m][e + 2] = __int_as_float(0x7fc00000);
        }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (bad[h] && i == 0) {
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 18 * D + ((tk + 8 * h) * NG + g) * 2), "h"(static_cast<uint16_t>(0)) : "memory");
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 19 * D + (g * kKvBlock + tk + 8 * h) * 2), "h"(static_cast<uint16_t>(0)) : "memory");
        }
    }
  }
  // the stage's next content comes by an asynchronous copy: it is ordered after these stores
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// The piece of unit u that begins at position from + n of the warp whose range is [from, to).
template <int D, int NT, class A>
__device__ __forceinline__ void set_piece(const A& a, const Unit& u, Piece<8 * NT>& p, int64_t from, int64_t to, int n) {
  constexpr int RB = 8 * NT, kStepTokens = step_blocks(D) * kKvBlock;
  const int lane = threadIdx.x & 31;
  const int64_t x = from + n;
  const int64_t base = u.rq.L - u.rq.T, row0 = u.rg * RB;
  const int64_t left = u.rq.T * a.group - row0, rows = left < RB ? left : RB;
  __syncwarp();                                                  // the previous piece is read out
  if (lane == 0) {
    p.q0 = u.rq.q0;
    p.row0 = row0;
    p.T = u.rq.T;
    p.start = u.start;
    p.n = u.n;
    p.cost = u.cost;
    p.h = u.h;
    p.rows = static_cast<int>(rows);
    const int64_t pos_first = base + quot(row0, a.group), pos_last = base + quot(row0 + rows - 1, a.group);
    // the last position that some row does not see
    const int64_t hidden = A::kSee == kOwn ? u.rq.low - 1 : A::kSee == kCausal && a.window > 0 ? pos_last - a.window : -1;
    p.first_full = hidden < 0 ? 0 : static_cast<int>(hidden / kStepTokens + 1);
    if constexpr (A::kSee == kAll) p.end_full = static_cast<int>(u.rq.L / kStepTokens);
    else p.end_full = pos_first < 0 ? 0 : static_cast<int>((pos_first + 1) / kStepTokens);
    if constexpr (A::kSee == kOwn) p.split = u.rq.low > 0;
    else if constexpr (A::kSee == kAll) p.split = a.pass != 0;
    else p.split = false;
    p.step0 = static_cast<int>(u.first + (x - u.start) - n);
    const int64_t end = u.start + u.n < to ? u.start + u.n : to;
    p.end = static_cast<int>(end - from);
    p.whole = x == u.start && end == u.start + u.n;
  }
  if (lane < RB) {
    const int64_t pos = base + quot(row0 + lane, a.group);
    p.hi[lane] = static_cast<int>(A::kSee != kAll && pos < u.rq.L ? pos : u.rq.L - 1);
    if constexpr (A::kSee == kOwn) p.lo[lane] = static_cast<int>(u.rq.low - 1);
    else p.lo[lane] = static_cast<int>(A::kSee == kCausal && a.window > 0 && pos - a.window > -1 ? pos - a.window : -1);
  }
  __syncwarp();
}

// The parts of unit u, cut between CTAs c0..c1, joined by the CTA that posted
// last, in the order of the CTAs.  `ring` is free.
template <int D, int NT, typename Out, class A>
__device__ __forceinline__ void join_parts(const A& a, Smem<D, NT, A::kSee>& sm, const Cut& u, int c0, int c1) {
  constexpr int RB = 8 * NT, kBatch = 10;
  constexpr int64_t kPitch = RB * (D + 2);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, parts = c1 - c0 + 1, rows = u.rows;
  auto part = [&](int c) { return a.partial + (2 * (c0 + c) + (c == 0 ? 1 : 0)) * kPitch; };
  float2* ml = reinterpret_cast<float2*>(sm.ring);             // [parts][RB]
  float2* total = ml + kKvMaxCtas * RB;                        // [RB]
  static_assert(sizeof(float2) * (kKvMaxCtas + 1) * RB <= sizeof(sm.ring));
  // items of 4 channels, each by `ways` threads (a power of two) that take every ways-th part
  const int items = rows * (D / 4);
  int ways = 1;
  while (2 * ways * items <= kThreads) ways *= 2;
  __syncthreads();
  for (int j = tid; j < parts * RB; j += kThreads)
    if (j % RB < rows) ml[j] = __ldcg(reinterpret_cast<const float2*>(part(j / RB) + RB * D) + j % RB);
#pragma unroll 1
  for (int j0 = 0; j0 < items * ways; j0 += kThreads) {
    const int j = j0 + tid, way = j & (ways - 1), item = j / ways, r = item / (D / 4);
    const bool have = item < items;
    float4 v[kBatch], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (have && way + k * ways < parts) v[k] = __ldcg(reinterpret_cast<const float4*>(part(way + k * ways)) + item);
    if (j0 == 0) {                                              // the weights, while the first loads are under way
      __syncthreads();
      for (int q = warp; q < rows; q += kWarps) {
        float m = kRefNone, l = 0.f;
        for (int c = lane; c < parts; c += 32) m = fmaxf(m, ml[c * RB + q].x);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        for (int c = lane; c < parts; c += 32) {
          const float2 w = ml[c * RB + q];
          const float f = ex2(w.x - m);
          ml[c * RB + q].x = f;
          l = fmaf(f, w.y, l);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        if (lane == 0) total[q] = make_float2(m, l);
      }
      __syncthreads();
    }
#pragma unroll 1
    for (int c = way;;) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (have && c + k * ways < parts) {
          const float f = ml[(c + k * ways) * RB + r].x;
          o.x = fmaf(f, v[k].x, o.x), o.y = fmaf(f, v[k].y, o.y), o.z = fmaf(f, v[k].z, o.z), o.w = fmaf(f, v[k].w, o.w);
        }
      c += kBatch * ways;
      if (c >= parts) break;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (have && c + k * ways < parts) v[k] = __ldcg(reinterpret_cast<const float4*>(part(c + k * ways)) + item);
    }
    // the ways of an item are neighbouring lanes: a fixed tree
    for (int x = 1; x < ways && x < 32; x <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
    }
    if (have && way == 0) {
      wait_first_pass(a);
      const float2 t = total[r];
      const int64_t at = out_row(a, u.q0, u.h, u.row0 + r);
      const RowScale sc = row_scale(a, u.split, at, t.x, t.y, (item & (D / 4 - 1)) == 0);
      const int64_t d = at * D + (item & (D / 4 - 1)) * 4;
      const float sums[4] = {o.x, o.y, o.z, o.w};
      put_row<Out, 4>(a, u.split, sc, [&](int k) { return d + k; }, [&](int k) { return t.y == 0.f ? 0.f : sums[k]; });
    }
  }
}

template <int D, int NT, typename Out, int SEE>
__global__ void __launch_bounds__(kThreads, D == 256 || NT > 1 ? 1 : 2) attention_kernel(const AttnArgsOf<SEE> a) {
  constexpr int RB = 8 * NT, S = ring_stages(D), SB = step_blocks(D), BB = kv_block_bytes(D), NG = D / 32;
  constexpr int kRegs = NT * (D / 16) * 4;                       // a lane's share of a warp's sums
  // blocks of a step taken together, as far as the registers reach
  constexpr int NB = D == 64 || (D == 128 && NT == 1) ? 2 : 1;
  static_assert(D == 256 || NT > 1 || sizeof(Smem<D, NT, SEE>) <= 113 * 1024);      // two CTAs per SM
  static_assert(kRegs * 128 <= S * stage_bytes(D));              // a warp's sums fit its ring
  extern __shared__ __align__(128) uint8_t smem[];
  Smem<D, NT, SEE>& sm = *reinterpret_cast<Smem<D, NT, SEE>*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (lane < S) {
    mbar_init(&sm.full[warp][lane], 1);
    fence_barrier_init();
  }
  if (lane < 2) sm.cut[2 * warp + lane].start = -1;
  if (tid == 0) sm.stopped = 0;
  if constexpr (SEE == kCausal) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else if (a.pass != 2) {
    // the second pass may start beside this one, once what was before both is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.pass == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }

  const Plan pl = make_plan<step_blocks(D), RB>(a, sm.prefix, sm.cost, sm.longest, sm.lower);
  if (pl.total == 0 || blockIdx.x >= pl.ctas) {
    wait_first_pass(a);
    return;
  }
  if (tid < 2) (tid ? sm.end : sm.begin) = bound<step_blocks(D), RB>(a, pl, blockIdx.x + tid);
  __syncthreads();
  if (sm.begin >= sm.end) {
    wait_first_pass(a);
    return;
  }
  const int steps = static_cast<int>(sm.end - sm.begin);
  const int first = static_cast<int>(static_cast<int64_t>(steps) * warp / kWarps);       // this warp's steps of the CTA's
  const int mine = static_cast<int>(static_cast<int64_t>(steps) * (warp + 1) / kWarps) - first;

  // The blocks of the warp's steps `from` .. +31 (step `from` lies in unit u); nullptr: nothing to copy.
  auto look_up = [&](int from, Unit u) {
    if (from + lane < mine) {
      const int64_t x = sm.begin + first + from + lane;
      if (x >= u.start + u.n) u = find_unit<step_blocks(D), RB>(a, pl, x);
#pragma unroll
      for (int j = 0; j < SB; ++j) {
        const int64_t blk = (u.first + (x - u.start)) * SB + j;
        const uint8_t* at = nullptr;
        if (blk * kKvBlock < u.rq.L && (blk + 1) * kKvBlock > first_visible(a, u.rq)) {
          at = kv_block_ptr(a.pool, a.kb, D, table_row(a, u.b), u.h, blk);
          if (at == nullptr) atomicOr(a.err, kErrIndex);
        }
        sm.src[warp][lane][j] = at;
      }
    }
    __syncwarp();
  };
  // Send the copies of the warp's step n into its stage.
  auto fetch = [&](int n) {
    if (lane == 0) {
      const int stage = n % S;
      const uint8_t* at[SB];
      uint32_t bytes = 0;
#pragma unroll
      for (int j = 0; j < SB; ++j) {
        at[j] = sm.src[warp][n & 31][j];
        bytes += at[j] != nullptr ? BB : 0;
      }
      mbar_arrive_expect_tx(&sm.full[warp][stage], bytes);
#pragma unroll
      for (int j = 0; j < SB; ++j)
        if (at[j] != nullptr) bulk_g2s(sm.ring[warp][stage] + j * BB, at[j], BB, &sm.full[warp][stage]);
    }
    __syncwarp();
  };
  if (mine > 0) {
    const Unit u = find_unit<step_blocks(D), RB>(a, pl, sm.begin + first);
    look_up(0, u);
    for (int n = 0; n < S && n < mine; ++n) fetch(n);
    set_piece<D, NT>(a, u, sm.piece[warp], sm.begin + first, sm.begin + first + mine, 0);
  }

  State<D, NT> st;
  const int i = lane & 3, tk = lane >> 2;
  Piece<RB>& p = sm.piece[warp];
  bool ok = true;
  for (int n = 0; n < mine;) {
    if (n > 0) set_piece<D, NT>(a, find_unit<step_blocks(D), RB>(a, pl, sm.begin + first + n), p, sm.begin + first, sm.begin + first + mine, n);
    load_q<D, NT>(a, p, st);
    reset<D, NT>(st);
    for (const int end = p.end; n < end; ++n) {
      const int stage = n % S;
      if (!mbar_wait_bounded(&sm.full[warp][stage], (n / S) & 1)) ok = false;
      if (!__all_sync(0xffffffffu, ok)) break;
      const int step = p.step0 + n;
      const uint32_t addr = smem_u32(sm.ring[warp][stage]);
      const bool full = step >= p.first_full && step < p.end_full;
#pragma unroll
      for (int j = 0; j < SB; j += NB) {
        uint32_t seen[NB] = {};
        if (!full) {
#pragma unroll
          for (int m = 0; m < NB; ++m) {
            const int blk = step * SB + j + m;
            seen[m] = seen_bits<NT>(p, blk);
            clear_hidden<D, NT>(st, p, addr + (j + m) * BB, blk * kKvBlock, seen[m]);
          }
        }
        block_step<D, NT, NB>(st, addr + j * BB, full, seen);
      }
      __syncwarp();                                               // the stage is read out
      if (n + S < mine) {
        if (((n + S) & 31) == 0) look_up(n + S, find_unit<step_blocks(D), RB>(a, pl, sm.begin + first + n + S));
        fetch(n + S);
      }
    }
    if (!__all_sync(0xffffffffu, ok)) {
      // a wait gave up: the copies under way land before the CTA leaves
      if (lane == 0) {
        sm.stopped = 1;
        atomicOr(a.err, kErrTimeout);
      }
      for (int m = n; m < n + S && m < mine; ++m) mbar_wait_bounded(&sm.full[warp][m % S], (m / S) & 1);
      break;
    }
    // the sums in the values' own units, the totals complete in every lane
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float2 back = make_float2(inv_pow2(st.fs[t].x), inv_pow2(st.fs[t].y));
#pragma unroll
      for (int o = 16; o > 2; o >>= 1) {
        st.l[t].x += __shfl_xor_sync(0xffffffffu, st.l[t].x, o);
        st.l[t].y += __shfl_xor_sync(0xffffffffu, st.l[t].y, o);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float z0 = __shfl_sync(0xffffffffu, st.corr[t][0], 4 * g + i), z1 = __shfl_sync(0xffffffffu, st.corr[t][1], 4 * g + i);
#pragma unroll
        for (int m = 2 * g; m < 2 * g + 2; ++m) {
          st.o[t][m][0] = fmaf(st.o[t][m][0], back.x, z0);
          st.o[t][m][1] = fmaf(st.o[t][m][1], back.y, z1);
          st.o[t][m][2] = fmaf(st.o[t][m][2], 0.0625f * back.x, z0);
          st.o[t][m][3] = fmaf(st.o[t][m][3], 0.0625f * back.y, z1);
        }
      }
    }
    if (p.whole) {
      wait_first_pass(a);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * t + 2 * i + e;
          if (r < p.rows) {
            const float l = e ? st.l[t].y : st.l[t].x;
            const int64_t at = out_row(a, p.q0, p.h, p.row0 + r);
            const RowScale sc = row_scale(a, p.split, at, e ? st.ref[t].y : st.ref[t].x, l, tk == 0);
            put_row<Out, D / 8>(a, p.split, sc, [&](int k) { return at * D + 8 * k + tk; },
                                [&](int k) { return l == 0.f ? 0.f : st.o[t][k >> 1][e + 2 * (k & 1)]; });
          }
        }
    } else {
      // a part: of the unit the warp began with (it goes on with others) or ended with
      const int which = n < mine ? 0 : 1;
      float* to = which ? reinterpret_cast<float*>(sm.ring[warp]) + lane
                        : a.stash + (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * (RB * D) + lane;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) to[32 * ((t * (D / 16) + m) * 4 + e)] = st.o[t][m][e];
        if (tk == 0) {
          sm.ml[2 * warp + which][8 * t + 2 * i] = make_float2(st.ref[t].x, st.l[t].x);
          sm.ml[2 * warp + which][8 * t + 2 * i + 1] = make_float2(st.ref[t].y, st.l[t].y);
        }
      }
      if (lane == 0) sm.cut[2 * warp + which] = {p.q0, p.row0, p.start, p.n, p.cost, p.h, p.rows, p.split};
    }
  }
  __syncthreads();
  if (sm.stopped) {
    wait_first_pass(a);
    return;
  }

  // Weights of the parts: entry c, row r against the largest reference among
  // the entries of the same unit.
  for (int j = tid; j < 2 * kWarps * RB; j += kThreads) {
    const int c = j / RB, r = j % RB;
    const int64_t unit = sm.cut[c].start;
    float m = kRefNone, l = 0.f;
#pragma unroll 4
    for (int o = 0; o < 2 * kWarps; ++o)
      if (sm.cut[o].start == unit && unit >= 0) m = fmaxf(m, sm.ml[o][r].x);
#pragma unroll 4
    for (int o = 0; o < 2 * kWarps; ++o)
      if (sm.cut[o].start == unit && unit >= 0) l = fmaf(ex2(sm.ml[o][r].x - m), sm.ml[o][r].y, l);
    sm.total[c][r] = make_float2(m, l);
  }
  // the entries with a part, and those that begin a unit
  const int64_t mine_at = lane < 2 * kWarps ? sm.cut[lane].start : -1;
  const uint32_t parts = __ballot_sync(0xffffffffu, mine_at >= 0), below = parts & ((1u << lane) - 1);
  const int64_t before = __shfl_sync(0xffffffffu, mine_at, below ? 31 - __clz(below) : lane);
  uint32_t begins = __ballot_sync(0xffffffffu, mine_at >= 0 && (below == 0 || before != mine_at));
  __syncthreads();
  int edge[2] = {-1, -1};                                         // entries of units cut between CTAs: begun before this one, going on after it
  constexpr int kEach = kRegs * 32 / kThreads;                    // a thread's places of the sums: register warp%4 + ..., lane
  const int e = warp & 3, d0 = 16 * (warp >> 2) + tk + 8 * (e >> 1);     // channels d0 + 32 j of rows row, row + 8
  const int row = 2 * i + (e & 1);
#pragma unroll 1
  while (begins != 0) {
    const int e0 = __ffs(begins) - 1;
    begins &= begins - 1;
    uint32_t left = parts & ~((1u << e0) - 1) & (begins ? (begins & (0u - begins)) - 1 : ~0u);
    const Cut& u = sm.cut[e0];
    const bool inside = u.start >= sm.begin && u.start + u.n <= sm.end;
    const int which = u.start >= sm.begin ? 1 : 0;
    if (!inside) edge[which] = e0;
    float o[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) o[j] = 0.f;
#pragma unroll 1
    for (; left != 0; left &= left - 1) {
      const int c = __ffs(left) - 1;
      const float* from = c & 1 ? reinterpret_cast<const float*>(sm.ring[c >> 1])
                                : a.stash + (static_cast<int64_t>(blockIdx.x) * kWarps + (c >> 1)) * (RB * D);
      float x[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) x[j] = from[tid + kThreads * j];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f = ex2(sm.ml[c][row + 8 * t].x - sm.total[c][row + 8 * t].x);
#pragma unroll
        for (int j = 0; j < kEach / NT; ++j) o[t * (kEach / NT) + j] = fmaf(f, x[t * (kEach / NT) + j], o[t * (kEach / NT) + j]);
      }
    }
    float* part = a.partial + static_cast<int64_t>(2 * blockIdx.x + which) * RB * (D + 2);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = row + 8 * t;
      if (r >= u.rows) break;
      const float2 v = sm.total[e0][r];
      const bool head = e < 2 && warp < 4 && tk == 0;             // one thread per row
      if (inside) {
        wait_first_pass(a);
        const int64_t at = out_row(a, u.q0, u.h, u.row0 + r);
        const RowScale sc = row_scale(a, u.split, at, v.x, v.y, head);
        put_row<Out, kEach / NT>(a, u.split, sc, [&](int j) { return at * D + d0 + 32 * j; },
                                 [&](int j) { return v.y == 0.f ? 0.f : o[t * (kEach / NT) + j]; });
      } else {
#pragma unroll
        for (int j = 0; j < kEach / NT; ++j) __stcg(part + r * D + d0 + 32 * j, o[t * (kEach / NT) + j]);
        if (head) __stcg(reinterpret_cast<float2*>(part + RB * D) + r, v);
      }
    }
  }
  if (edge[0] < 0 && edge[1] < 0) {
    wait_first_pass(a);
    return;
  }
  __syncthreads();
  // the CTAs with a part of a unit: those whose shares begin where it may be cut, and the one before
  if (tid < 2 && edge[tid] >= 0) {
    const Cut& u = sm.cut[edge[tid]];
    const int c0 = share_of(pl, u.cost + kUnitCost + cut_steps<RB> - 1), c1 = share_of(pl, u.cost + kUnitCost + u.n - cut_steps<RB>);
    // release: the CTA's parts, stored before the barrier, come first; acquire: the last one sees the others'
    uint32_t count;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(count) : "l"(a.counters + c0) : "memory");
    const bool last = count == static_cast<uint32_t>(c1 - c0);
    if (last) a.counters[c0] = 0;
    sm.joins[tid] = last ? c0 << 16 | c1 : -1;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k)
    if (edge[k] >= 0 && sm.joins[k] >= 0) join_parts<D, NT, Out>(a, sm, sm.cut[edge[k]], sm.joins[k] >> 16, sm.joins[k] & 0xFFFF);
  wait_first_pass(a);
}

template <int D, int NT, typename Out, int SEE>
cudaError_t launch_variant(const AttnArgsOf<SEE>& a, int grid, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(attention_kernel<D, NT, Out, SEE>);
  cudaError_t e = set_max_dynamic_smem(f);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem<D, NT, SEE>);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_kernel<D, NT, Out, SEE>, a);
}

}  // namespace

template <int SEE>
cudaError_t launch_attention_rows(int D, bool two, const AttnArgsOf<SEE>& a, int out_f32, const DeviceInfo& info, cudaStream_t s) {
  const int per_sm = D == 256 || two ? 1 : 2;
  const int most = two ? kKvMaxCtas / 2 : kKvMaxCtas;
  const int grid = info.sms * per_sm < most ? info.sms * per_sm : most;
#define Q4NX_ATTN(DD)                                                                                                       \
  case DD:                                                                                                                  \
    return two ? (out_f32 ? launch_variant<DD, 2, float, SEE>(a, grid, s) : launch_variant<DD, 2, uint16_t, SEE>(a, grid, s)) \
               : (out_f32 ? launch_variant<DD, 1, float, SEE>(a, grid, s) : launch_variant<DD, 1, uint16_t, SEE>(a, grid, s));
  switch (D) {
    Q4NX_ATTN(64)
    Q4NX_ATTN(128)
    Q4NX_ATTN(256)
    default: return cudaErrorInvalidValue;
  }
#undef Q4NX_ATTN
}

}  // namespace q4nx
