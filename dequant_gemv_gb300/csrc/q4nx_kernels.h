// q4nx_kernels.h -- host-side launchers of the Q4NX kernels (internal to libq4nx.so).
// The C ABI in include/q4nx.h validates arguments and then calls these.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace q4nx {

struct DeviceInfo {
  int sms = 0;
  int max_smem_optin = 0;      // dynamic shared memory one CTA may opt in to
  int smem_two_per_sm = 0;     // the most dynamic shared memory a CTA may use with two CTAs on one SM
};
// Properties of the current device (cached per device ordinal).
cudaError_t device_info(DeviceInfo* out);

// Raise a kernel's dynamic shared-memory limit to the device maximum once per
// (device, kernel).
cudaError_t set_max_dynamic_smem(const void* func);

// ---- GEMV (M = 1), a batch of independent items of one kind per launch ----
constexpr int kMaxGemvItems = 256;
struct GemvItem {
  const void* chunks;
  const void* x;
  void* y;
  int64_t TR, TC;
};
struct GemvPlan {
  int warps = 0;       // warps per CTA, each owning a contiguous part of the CTA's chunks
  int stages = 0;      // ring stages per warp
  int grid = 0;        // CTAs, each owning a contiguous range of chunks
  size_t smem = 0;     // dynamic shared memory bytes
  int xslots = 0;      // x-slice cache slots, one per slice holding every token (4-bit kinds)
  int quarter = 0;     // the units are quarters of chunks (small 4-bit launches, one token)
};
// tc: tile columns of the launch's one weight (several tokens), else 0
bool gemv_plan(int kind, int64_t total_chunks, const DeviceInfo& info, GemvPlan* plan, int tokens, int64_t tc = 0);
uint64_t gemv_workspace_bytes(int64_t total_tile_rows, int64_t total_chunks, int tokens = 1);
cudaError_t launch_gemv_batch(int kind, const GemvItem* items, int n, int out_f32, void* workspace,
                              const DeviceInfo& info, cudaStream_t s);

// GEMV of one item fused with top-1: the largest fp32 output (ties: lowest
// row; a NaN output wins, the first one), y not written.  Writes the row to
// *idx and/or the 64-bit key (top bit flipped, see q4nx.h) to *key, the rows
// numbered from row_base.  The workspace's bytes 4..15 hold the launch's
// top-1 words (zero between launches).
cudaError_t launch_gemv_top1(int kind, const GemvItem& item, int32_t* idx, int64_t* key, uint32_t row_base,
                             void* workspace, const DeviceInfo& info, cudaStream_t s);

// ---- GEMV of one weight against M tokens (X [M][cols], Y [M][rows]) ----
// Each chunk is read once for all M tokens.  M up to gemv_max_tokens(kind),
// the M up to which this beats the tensor-core GEMM on GB300 (measured: two
// tokens for q4_1, one for Q8, whose float path costs more per token); Q4_K
// has no tensor-core path, so it goes to four.  `workspace`:
// gemv_workspace_bytes(.., .., 4) bytes, zero-filled and left so; `err`: the
// error word to report a failed wait in.
constexpr int kGemvTokensQ41 = 2, kGemvTokensQ4K = 4, kGemvTokensQ8 = 1, kGemvTokensMax = 4;
int gemv_max_tokens(int kind);
// `ep`: what is done to the sums before they are stored (q4nx_epilogue.cuh).
struct Epilogue;
cudaError_t launch_gemv_tokens(int kind, const GemvItem& item, int M, int out_f32, uint32_t* err, void* workspace,
                               const DeviceInfo& info, cudaStream_t s, const Epilogue* ep = nullptr);

// ---- standalone decode ----
cudaError_t launch_decode(int kind, const void* chunks, int64_t TR, int64_t TC, void* out, cudaStream_t s);

// ---- Q4_K -> q4_1 repack ----
cudaError_t launch_repack_q4k(const void* in, int64_t TR, int64_t TC, void* out, cudaStream_t s);

// ---- GGUF-type tensor -> q4_1 chunks ----
enum : int { kSrcQ4_0 = 1, kSrcQ4_1 = 2, kSrcQ8_0 = 3, kSrcF32 = 4, kSrcF16 = 5, kSrcBF16 = 6 };
int pack_src_bytes_per_32(int src_type);        // 0 for an unknown type
cudaError_t launch_pack_q4_1(int src_type, const void* src, int64_t TR, int64_t TC, void* out, cudaStream_t s);

// ---- top-1 ----
cudaError_t launch_argmax(const float* logits, int M, int64_t V, int32_t* idx, cudaStream_t s);

// ---- GEMM (M <= 64, tcgen05) ----
bool gemm_supports(int kind);
uint64_t gemm_workspace_bytes(int64_t TR, int64_t TC, int M);
// after_wait: a dependent launch that starts early finds what the grids before the GEMM wrote
cudaError_t launch_gemm(int kind, const void* chunks, int64_t TR, int64_t TC, const void* X, int M, void* Y,
                        int out_f32, void* workspace, cudaStream_t s, bool after_wait = false, const Epilogue* ep = nullptr);

// ---- 4-bit key/value cache and the attention that reads it (q4nx_kv.cuh) ----
struct KvPool;
struct KvBatch;
constexpr int kKvMaxBatch = 1024;                 // requests per call
constexpr int kKvMaxCtas = 304;                   // CTAs of an attention launch, at most
cudaError_t launch_kv_append(int D, const KvPool& p, const KvBatch& kb, const void* k, const void* v, int64_t stride,
                             uint32_t* err, cudaStream_t s);
struct RotaryCall {
  const uint16_t *q, *k, *v;   // bf16 rows of tokens
  uint16_t* q_out;
  int64_t q_stride, q_out_stride, kv_stride;   // elements from token to token
  const float2* table;         // [positions][half] cosine and sine
  int64_t positions;
  int half;                    // pairs of channels that are turned
  int interleaved;             // pairs are (2j, 2j + 1), else (j, j + half)
  int heads;                   // query heads; 0: no queries
  uint32_t* err;
};
cudaError_t launch_kv_append_rotary(int D, const KvPool& p, const KvBatch& kb, const RotaryCall& c, cudaStream_t s);
cudaError_t launch_kv_read(int D, const KvPool& p, const KvBatch& kb, void* k, void* v, int out_f32, uint32_t* err,
                           cudaStream_t s);
uint64_t attention_workspace_bytes(int D);
cudaError_t launch_attention(int D, const KvPool& pool, const KvBatch& kb, const void* q, int64_t q_stride, int heads,
                             float scale, int64_t window, void* out, int out_f32, float* lse, void* workspace,
                             const DeviceInfo& info, cudaStream_t s);

cudaError_t launch_attention_cross(int D, const KvPool& pool, const KvBatch& kb, const void* q, int64_t q_stride, int heads,
                                   float scale, void* out, int out_f32, float* lse, void* workspace, const DeviceInfo& info,
                                   cudaStream_t s);
// Requests first[g] .. first[g + 1] - 1 share their first shared[g] positions (q4nx_attention.cu).
uint64_t attention_shared_scratch(int D, int64_t tokens, int heads);
cudaError_t launch_attention_shared(int D, const KvPool& pool, const KvBatch& kb, const int32_t* first, const int32_t* shared,
                                    int groups, const void* q, int64_t q_stride, int heads, float scale, void* out,
                                    int out_f32, float* lse, void* workspace, void* scratch, const DeviceInfo& info,
                                    cudaStream_t s);

// ---- low-rank adapters beside a projection ----
struct LoraCall {
  const void *x, *a, *b;       // bf16 [M][K], [count][R][K], [count][N][R]
  const float* scale;          // [count]
  const int32_t* ids;          // [M]
  float* t;                    // scratch: lora_splits(K) * 64 * R numbers, then 64 pairs of int
  const float* base;           // the product with W, binary32 [M][N] (may be y)
  void* y;                     // [M][N]
  uint32_t* err;
  int64_t K, N;
  int M, R, count;
};
int lora_splits(int64_t K);     // parts into which shrink cuts the columns
// beside: behind the launch of the product (after_wait), while that runs
cudaError_t launch_lora_shrink(const LoraCall& c, const DeviceInfo& info, bool beside, cudaStream_t s);
cudaError_t launch_lora_expand(const LoraCall& c, int out_f32, cudaStream_t s);

// ---- log-probabilities ----
constexpr int kMaxTopLogprobs = 32;
struct LogprobsCall {
  const void* logits;
  int f32, M, top;
  int64_t V, stride;           // columns, elements between rows
  const int32_t* tokens;
  float *logprob, *entropy, *lse;   // NULL: not wanted
  int32_t* top_idx;
  float* top_lp;
};
cudaError_t launch_logprobs(const LogprobsCall& c, const DeviceInfo& info, cudaStream_t s);

// Workspace layout shared by the GEMV launcher and kernel.
constexpr uint64_t kWsErrBytes = 16;              // error word (+ padding)
constexpr int kMaxCtas = 1024;                    // upper bound of CTAs per GEMV launch
__host__ __device__ inline uint64_t align16(uint64_t v) { return (v + 15) & ~uint64_t(15); }

}  // namespace q4nx
