// q4nx_serve_api.cu -- the C ABI of the operators around the products in a
// decode step (declared in include/q4nx.h): the 4-bit key/value cache and its
// attention, adapters beside a projection, log-probabilities.  As in
// q4nx_api.cu everything that the host can see is checked before any work is
// enqueued; numbers that live on the device (lengths, pages, adapter ids) are checked
// by the kernels, which skip what is out of range and report it in the
// workspace's error word.
#include <cstdint>

#include "../../include/q4nx.h"
#include "q4nx_checks.h"
#include "q4nx_kernels.h"
#include "q4nx_kv.cuh"

using namespace q4nx;

namespace {

int from_cuda(cudaError_t e) { return e == cudaSuccess ? Q4NX_OK : Q4NX_E_CUDA; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known_out(int t) { return t == Q4NX_OUT_BF16 || t == Q4NX_OUT_F32; }

int check_cache(const q4nx_kv_cache* c) {
  if (c == nullptr || c->pool_dev == nullptr) return Q4NX_E_NULL;
  if (c->reserved != 0) return Q4NX_E_KIND;
  const uint64_t page = q4nx_kv_page_bytes(c->head_dim, c->kv_heads, c->page_tokens);
  if (page == 0 || c->pages <= 0 || c->pages > INT32_MAX) return Q4NX_E_SHAPE;
  if (c->bytes / page < static_cast<uint64_t>(c->pages)) return Q4NX_E_SHORT;
  if (!aligned16(c->pool_dev)) return Q4NX_E_ALIGN;
  return Q4NX_OK;
}

int check_batch(const q4nx_kv_batch* b) {
  if (b == nullptr || b->q_start_dev == nullptr || b->lens_dev == nullptr || b->table_dev == nullptr) return Q4NX_E_NULL;
  if (b->batch < 1 || b->batch > kKvMaxBatch || b->table_cols < 1 || b->tokens < 0 || b->tokens > INT32_MAX) return Q4NX_E_SHAPE;
  if (!aligned(b->q_start_dev, 4) || !aligned(b->lens_dev, 4) || !aligned(b->table_dev, 4)) return Q4NX_E_ALIGN;
  return Q4NX_OK;
}

int check_workspace(const void* ws, uint64_t bytes, uint64_t need) {
  if (ws == nullptr || bytes < need) return Q4NX_E_WORKSPACE;
  return aligned16(ws) ? Q4NX_OK : Q4NX_E_ALIGN;
}

KvPool pool_of(const q4nx_kv_cache* c) {
  KvPool p;
  p.pool = static_cast<uint8_t*>(c->pool_dev);
  p.pages = c->pages;
  p.kv_heads = c->kv_heads;
  p.page_blocks = c->page_tokens / kKvBlock;
  return p;
}
KvBatch batch_of(const q4nx_kv_batch* b) {
  KvBatch k;
  k.q_start = b->q_start_dev;
  k.lens = b->lens_dev;
  k.table = b->table_dev;
  k.batch = b->batch;
  k.table_cols = b->table_cols;
  k.tokens = b->tokens;
  return k;
}

constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxStride = int64_t(1) << 40;      // elements between rows: products of it stay in 64 bits

// 32-bit words of the adapters' inner products and of the tokens in their order
uint64_t lora_t(int64_t cols) { return static_cast<uint64_t>(lora_splits(cols)) * 64 * 128 + 128; }
bool known_rank(int r) { return r == 8 || r == 16 || r == 32 || r == 64 || r == 128; }

}  // namespace

extern "C" {

uint64_t q4nx_kv_page_bytes(int head_dim, int kv_heads, int page_tokens) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  if (kv_heads < 1 || kv_heads > kMaxHeads || page_tokens < kKvBlock || page_tokens % kKvBlock != 0) return 0;
  return static_cast<uint64_t>(page_tokens / kKvBlock) * kv_heads * kv_block_bytes(head_dim);
}

uint64_t q4nx_kv_workspace(const q4nx_kv_cache* cache) {
  if (cache == nullptr || q4nx_kv_page_bytes(cache->head_dim, cache->kv_heads, cache->page_tokens) == 0) return 0;
  return attention_workspace_bytes(cache->head_dim);
}

int q4nx_kv_append(const q4nx_kv_cache* cache, const q4nx_kv_batch* batch, const void* k_dev, const void* v_dev,
                   int64_t kv_stride, void* workspace_dev, uint64_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st == Q4NX_OK) st = check_batch(batch);
  if (st) return st;
  if (k_dev == nullptr || v_dev == nullptr) return Q4NX_E_NULL;
  if (kv_stride < static_cast<int64_t>(cache->kv_heads) * cache->head_dim || kv_stride > kMaxStride) return Q4NX_E_SHAPE;
  if (!aligned16(k_dev) || !aligned16(v_dev) || kv_stride % 8 != 0) return Q4NX_E_ALIGN;
  if ((st = check_workspace(workspace_dev, workspace_bytes, q4nx_kv_workspace(cache)))) return st;
  if (batch->tokens == 0) return Q4NX_OK;
  return from_cuda(launch_kv_append(cache->head_dim, pool_of(cache), batch_of(batch), k_dev, v_dev, kv_stride,
                                    static_cast<uint32_t*>(workspace_dev), static_cast<cudaStream_t>(stream)));
}

int q4nx_kv_read(const q4nx_kv_cache* cache, const q4nx_kv_batch* batch, void* k_dev, void* v_dev, int out_dtype,
                 void* workspace_dev, uint64_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st == Q4NX_OK) st = check_batch(batch);
  if (st) return st;
  if (k_dev == nullptr || v_dev == nullptr) return Q4NX_E_NULL;
  if (!known_out(out_dtype)) return Q4NX_E_DTYPE;
  if (!aligned16(k_dev) || !aligned16(v_dev)) return Q4NX_E_ALIGN;
  if ((st = check_workspace(workspace_dev, workspace_bytes, q4nx_kv_workspace(cache)))) return st;
  if (batch->tokens == 0) return Q4NX_OK;
  return from_cuda(launch_kv_read(cache->head_dim, pool_of(cache), batch_of(batch), k_dev, v_dev,
                                  out_dtype == Q4NX_OUT_F32, static_cast<uint32_t*>(workspace_dev),
                                  static_cast<cudaStream_t>(stream)));
}

int q4nx_kv_attention(const q4nx_kv_cache* cache, const q4nx_kv_batch* batch, const void* q_dev, int64_t q_stride,
                      int heads, float scale, int64_t window, void* out_dev, int out_dtype, float* lse_dev,
                      void* workspace_dev, uint64_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st == Q4NX_OK) st = check_batch(batch);
  if (st) return st;
  if (q_dev == nullptr || out_dev == nullptr) return Q4NX_E_NULL;
  if (heads < 1 || heads > kMaxHeads || heads % cache->kv_heads != 0) return Q4NX_E_SHAPE;
  if (q_stride < static_cast<int64_t>(heads) * cache->head_dim || q_stride > kMaxStride || window < 0) return Q4NX_E_SHAPE;
  if (!known_out(out_dtype)) return Q4NX_E_DTYPE;
  if (!aligned16(q_dev) || !aligned16(out_dev) || q_stride % 8 != 0 || !aligned(lse_dev, 4)) return Q4NX_E_ALIGN;
  if ((st = check_workspace(workspace_dev, workspace_bytes, q4nx_kv_workspace(cache)))) return st;
  if (batch->tokens == 0) return Q4NX_OK;
  DeviceInfo info;
  if (device_info(&info) != cudaSuccess) return Q4NX_E_CUDA;
  return from_cuda(launch_attention(cache->head_dim, pool_of(cache), batch_of(batch), q_dev, q_stride, heads, scale, window,
                                    out_dev, out_dtype == Q4NX_OUT_F32, lse_dev, workspace_dev, info,
                                    static_cast<cudaStream_t>(stream)));
}

uint64_t q4nx_gemm_lora_scratch(const q4nx_weight* w, int M) {
  if (w == nullptr || check_grid(w->rows, w->cols) != Q4NX_OK || M < 1 || M > 64) return 0;
  return lora_t(w->cols) * 4 + static_cast<uint64_t>(M) * static_cast<uint64_t>(w->rows) * 4;
}

int q4nx_gemm_lora(const q4nx_weight* w, const void* X_dev, int M, const q4nx_adapters* ad, const int32_t* ids_dev,
                   void* Y_dev, int out_dtype, void* workspace_dev, uint64_t workspace_bytes, void* scratch_dev,
                   uint64_t scratch_bytes, void* stream) {
  int st = check_weight(w);
  if (st) return st;
  if (X_dev == nullptr || Y_dev == nullptr || ids_dev == nullptr || ad == nullptr || ad->a_dev == nullptr ||
      ad->b_dev == nullptr || ad->scale_dev == nullptr)
    return Q4NX_E_NULL;
  if (M < 1 || M > 64) return Q4NX_E_M;
  if (ad->count < 1 || !known_rank(ad->rank)) return Q4NX_E_SHAPE;
  const uint64_t row = static_cast<uint64_t>(ad->rank) * 2, pool = static_cast<uint64_t>(ad->count);
  if (ad->a_bytes / row / static_cast<uint64_t>(w->cols) < pool || ad->b_bytes / row / static_cast<uint64_t>(w->rows) < pool)
    return Q4NX_E_SHORT;
  if (!known_out(out_dtype)) return Q4NX_E_DTYPE;
  if (!aligned16(X_dev) || !aligned16(Y_dev) || !aligned16(ad->a_dev) || !aligned16(ad->b_dev) ||
      !aligned(ad->scale_dev, 4) || !aligned(ids_dev, 4))
    return Q4NX_E_ALIGN;
  if (M > gemv_max_tokens(w->kind) && !gemm_supports(w->kind)) return Q4NX_E_UNSUPPORTED;
  if ((st = check_workspace(workspace_dev, workspace_bytes, q4nx_gemm_workspace(w, M)))) return st;
  if ((st = check_workspace(scratch_dev, scratch_bytes, q4nx_gemm_lora_scratch(w, M)))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = out_dtype == Q4NX_OUT_F32;
  LoraCall c;
  c.x = X_dev;
  c.a = ad->a_dev;
  c.b = ad->b_dev;
  c.scale = ad->scale_dev;
  c.ids = ids_dev;
  c.t = static_cast<float*>(scratch_dev);
  float* base = f32 ? static_cast<float*>(Y_dev) : c.t + lora_t(w->cols);
  c.base = base;
  c.y = Y_dev;
  c.err = static_cast<uint32_t*>(workspace_dev);
  c.K = w->cols;
  c.N = w->rows;
  c.M = M;
  c.R = ad->rank;
  c.count = ad->count;
  DeviceInfo info;
  if (device_info(&info) != cudaSuccess) return Q4NX_E_CUDA;
  if (M > gemv_max_tokens(w->kind)) {
    // the tensor-core product leaves SMs free: shrink runs on them beside it
    if (launch_gemm(w->kind, w->chunks_dev, w->rows / 32, w->cols / 256, X_dev, M, base, 1, workspace_dev, s, true) != cudaSuccess ||
        launch_lora_shrink(c, info, true, s) != cudaSuccess)
      return Q4NX_E_CUDA;
  } else {
    if (launch_lora_shrink(c, info, false, s) != cudaSuccess) return Q4NX_E_CUDA;
    if ((st = q4nx_gemm_m64(w, X_dev, M, base, Q4NX_OUT_F32, workspace_dev, workspace_bytes, stream))) return st;
  }
  return from_cuda(launch_lora_expand(c, f32, s));
}

int q4nx_logprobs(const void* logits_dev, int dtype, int M, int64_t V, int64_t stride, const int32_t* tokens_dev, int top,
                  float* logprob_dev, float* entropy_dev, float* lse_dev, int32_t* top_idx_dev, float* top_logprob_dev,
                  void* stream) {
  if (logits_dev == nullptr || (logprob_dev != nullptr && tokens_dev == nullptr)) return Q4NX_E_NULL;
  if (M < 1 || M > 65535 || V < 1 || V > INT32_MAX || stride < V || stride > kMaxStride) return Q4NX_E_SHAPE;
  if (top < 0 || top > kMaxTopLogprobs || top > V) return Q4NX_E_SHAPE;
  if (top > 0 && (top_idx_dev == nullptr || top_logprob_dev == nullptr)) return Q4NX_E_NULL;
  if (!known_out(dtype)) return Q4NX_E_DTYPE;
  if (!aligned(logits_dev, dtype == Q4NX_OUT_F32 ? 4 : 2) || !aligned(tokens_dev, 4) || !aligned(logprob_dev, 4) ||
      !aligned(entropy_dev, 4) || !aligned(lse_dev, 4) || !aligned(top_idx_dev, 4) || !aligned(top_logprob_dev, 4))
    return Q4NX_E_ALIGN;
  DeviceInfo info;
  if (device_info(&info) != cudaSuccess) return Q4NX_E_CUDA;
  LogprobsCall c;
  c.logits = logits_dev;
  c.f32 = dtype == Q4NX_OUT_F32;
  c.M = M;
  c.top = top;
  c.V = V;
  c.stride = stride;
  c.tokens = tokens_dev;
  c.logprob = logprob_dev;
  c.entropy = entropy_dev;
  c.lse = lse_dev;
  c.top_idx = top_idx_dev;
  c.top_lp = top_logprob_dev;
  return from_cuda(launch_logprobs(c, info, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
