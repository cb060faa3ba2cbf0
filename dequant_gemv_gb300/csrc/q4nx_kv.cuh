// q4nx_kv.cuh -- the 4-bit key/value cache: block layout and request lookup,
// shared by the append / read kernels and the attention kernels.
//
// A value x of a group of 32 channels of one token is kept as
//   x ~ (code - 8) * scale + mid,   code in 0..15, scale and mid bf16.
// The middle of the 16 levels is stored instead of their lowest (the weights'
// q4_1 zero): it is small where the values straddle zero, so its bf16
// rounding is small, and the codes that meet it in a product are signed and
// centred, so that long sums stay near their result.
//
// The pool holds pages of `page_tokens` tokens (a multiple of 16), a page the
// kv heads one after another, a head its 16-token blocks one after another.
// A block is the unit of every copy (20*D bytes for D channels, contiguous:
// 0.625 bytes per value) and holds the operands of m16n8k16 matrix products in
// the order in which a warp's lanes want them; NG = D/32 groups:
//   0      K codes  [D/128 halves][16 tokens][4 i][words of groups 4*half..]  (D = 64: one half of 2 groups)
//          word (t, i, g): the codes of channels 32g + 8i .. +7 of token t;
//          nibble j holds channel 2j, nibble j + 4 channel 2j + 1 (j < 4)
//   8D     V codes  [D/64][32 lanes][4 words]; word (lane, mt = 4q + word):
//          channels d = 16mt + lane/4 and d + 8 of tokens 2i, 2i+1, 2i+8, 2i+9
//          (i = lane%4); byte 0 token 2i, byte 1 2i+8, byte 2 2i+1, byte 3 2i+9;
//          low nibble channel d, high nibble d + 8
//   16D    K scale bf16 [16][NG]    17D  K mid [16][NG]    18D  V scale [16][NG]    19D  V mid [NG][16]
// A byte never holds codes of two tokens, so tokens are appended without
// reading what is there.
#pragma once

#include <cstdint>

#include "q4nx_device.cuh"

namespace q4nx {

constexpr int kKvBlock = 16;                      // tokens per block
constexpr uint32_t kErrTimeout = 1, kErrIndex = 2;  // bits of a workspace's error word

__host__ __device__ constexpr int kv_block_bytes(int D) { return 20 * D; }

struct KvPool {
  uint8_t* pool;
  int64_t pages;
  int kv_heads;
  int page_blocks;        // 16-token blocks per page
};

// The requests of a call: tokens q_start[b] .. q_start[b+1] of the call are the
// last ones of request b, whose cache holds lens[b] tokens with them.
struct KvBatch {
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* table;   // [batch][table_cols] page of each page_tokens positions
  int batch, table_cols;
  int64_t tokens;
};

struct KvRequest {
  int64_t q0;             // first token of the call
  int64_t T, L;           // tokens of the call, tokens in the cache
  bool ok;
  int64_t low = 0;        // attention of a request's own part: its first position
};

// A request with its numbers checked: a length below 0 or beyond the table, or
// token ranges that do not lie in 0..tokens in order, make it empty (ok false).
__device__ __forceinline__ KvRequest kv_checked(const KvBatch& kb, int page_blocks, int64_t q0, int64_t q1, int64_t L) {
  KvRequest r = {};
  const int64_t cap = static_cast<int64_t>(kb.table_cols) * page_blocks * kKvBlock;
  r.ok = q0 >= 0 && q1 >= q0 && q1 <= kb.tokens && L >= 0 && L <= cap;
  r.q0 = r.ok ? q0 : 0;
  r.T = r.ok ? q1 - q0 : 0;
  r.L = r.ok ? L : 0;
  return r;
}
__device__ __forceinline__ KvRequest kv_request(const KvBatch& kb, int page_blocks, int b) {
  return kv_checked(kb, page_blocks, kb.q_start[b], kb.q_start[b + 1], kb.lens[b]);
}

// Reports the requests that kv_checked refuses; by a whole warp.  Many of them have
// no tokens that a warp of the append or read kernels would come by, so that a warp
// beyond those with work looks at all of them.
__device__ __forceinline__ void kv_report(const KvBatch& kb, int page_blocks, uint32_t* err) {
  for (int b = threadIdx.x & 31; b < kb.batch; b += 32)
    if (!kv_request(kb, page_blocks, b).ok) atomicOr(err, kErrIndex);
}

// Block `blk` (16 positions) of request b and kv head h, or NULL where the
// table names no page of the pool.
__device__ __forceinline__ uint8_t* kv_block_ptr(const KvPool& p, const KvBatch& kb, int D, int b, int h, int64_t blk) {
  const int64_t col = blk / p.page_blocks;
  const int32_t page = kb.table[static_cast<int64_t>(b) * kb.table_cols + col];
  if (page < 0 || page >= p.pages) return nullptr;
  const int64_t in_page = blk - col * p.page_blocks;
  return p.pool + ((static_cast<int64_t>(page) * p.kv_heads + h) * p.page_blocks + in_page) * kv_block_bytes(D);
}

// Offsets of one token's codes inside a block.
__device__ __forceinline__ int kv_k_word(int D, int t, int i, int g) {   // 32-bit word of channels 32g+8i..+7
  return D == 64 ? ((t * 4 + i) * 2 + g) * 4 : (g >> 2) * 1024 + ((t * 4 + i) * 4 + (g & 3)) * 4;
}
__device__ __forceinline__ int kv_v_byte(int D, int t, int mt, int r) {  // byte of channels 16mt+r and +8
  const int i = (t & 7) >> 1, lane = r * 4 + i;
  return 8 * D + ((mt >> 2) * 32 + lane) * 16 + (mt & 3) * 4 + (t >> 3) + 2 * (t & 1);
}

// The request that holds token `tok` of the call (b), or -1 where there is none;
// by a whole warp, in one round trip to memory for 32 requests (a binary
// search takes one for each of its steps).
__device__ __forceinline__ KvRequest kv_locate(const KvBatch& kb, int page_blocks, int64_t tok, int& b) {
  const int lane = threadIdx.x & 31;
  b = -1;
  for (int j0 = 0; j0 < kb.batch; j0 += 32) {
    const int j = j0 + lane;
    int32_t q0 = 0, q1 = 0, L = 0;
    if (j < kb.batch) q0 = kb.q_start[j], q1 = kb.q_start[j + 1], L = kb.lens[j];
    const uint32_t here = __ballot_sync(0xffffffffu, q0 <= tok && tok < q1);
    if (here == 0) continue;
    const int src = __ffs(here) - 1;
    b = j0 + src;
    return kv_checked(kb, page_blocks, __shfl_sync(0xffffffffu, q0, src), __shfl_sync(0xffffffffu, q1, src),
                      __shfl_sync(0xffffffffu, L, src));
  }
  return KvRequest{0, 0, 0, false};
}

}  // namespace q4nx
