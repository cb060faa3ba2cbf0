// q4nx_attention.cu -- attention over the 4-bit cache: which kernel a call takes, the
// workspace, and the kernel for few query rows, positions up to a row's own.
//
// Rows per request on average decide: a tile of 8, two tiles that share each block's
// decoding, or 256 rows on the tensor cores.  48 requests of 600 to 6000 tokens, 8 kv
// heads of 128: 16 rows by one tile after another 101, by two at once 88 us; 8 rows by one
// tile 65, by two 83.  One tile leaves registers for two CTAs per SM: 65 instead of 72 us
// with one (256 channels and two tiles do not).
//
// What the requests of a group share is attended to by the rows of all of them together, as
// if the group were one request with all its tokens: the cache's bytes are read and decoded
// once for the group instead of once for each request, and the rows are as many as
// the tensor cores want.  What a request has of its own is a second pass.  Each row's output
// of the first pass and its two softmax numbers stay in the caller's scratch, in binary32; the second pass
// joins them to its own when it writes a row.  It starts beside the first one and waits
// for it only then, so that the second plan, look-ups and first copies cost no time of their own.
//
// Shared (whole calls, against a floor by bytes): 48 requests behind 8191 positions, 32 query
// heads, 8 kv heads of 128: 59 us (4.7); cold and alone the requests' own 60 to 600 tokens take 24 and the prefix on the
// tensor cores 34; 16 requests behind 65537: 135 (14); 12 requests x 4 tokens, two groups behind 16001
// positions, 4 kv heads of 256: 83 (5.9), by passes of 16 rows over the prefix 108; 4 requests behind 300: 18, two
// plans, look-ups and joins.  Cross: 32 requests of 410 to 4097 positions: 37 us, 2.6 TB/s, as the kernel for few rows does.
#include "q4nx_attention_rows.cuh"

namespace q4nx {

template cudaError_t launch_attention_rows<kCausal>(int, bool, const AttnArgsOf<kCausal>&, int, const DeviceInfo&, cudaStream_t);

namespace {

// From so many query rows per request on, the tensor-core kernel.  It costs the same
// up to 128 rows, the other one a pass for each 16: one request of 16384 tokens, 8 kv
// heads of 128 channels: 64 rows 47 (there) and 49 us (tensor cores), 68 rows 53 and 49,
// 256 rows 115 and 57; 16 requests of 4096: 64 rows 119 and 137, 68 rows 143 and
// 139, 256 rows 401 and 172; 64 channels: 88 and 109, 104 and 109, 285 and 125 (with a join that took 3 us more).  Where every
// row sees everything (cross attention, prefixes) much the same, its two tiles sharing what few rows there
// are: one request of 65536, 64 rows 104 and 108, 128 rows 193 and 110; 64 channels: 78 and 87, 143 and 87.
// 256 channels, 4 kv heads, there alone: one request of 16384, 64 rows 53 and 53, 96 rows 62 and 51, 256 rows 119 and 83;
// 16 of 2048: 96 rows 101 and 101, 128 rows 125 and 105, 256 rows 222 and 171.  (Attention up to a row's own position stays with the other
// kernel at 256 channels, whose numbers are its documented ones.)
constexpr int kManyRows = 65;

// The workspace: the error word, a counter and a record per CTA and pass, then any
// content: per CTA two parts of 8 rows and one of each warp (half as many CTAs
// with twice the rows), or the parts of the kernel for many rows.  A second pass has its
// parts in the caller's scratch.
constexpr uint64_t kPassBytes = kKvMaxCtas * 4 + kKvMaxCtas * sizeof(Joined);
constexpr uint64_t kPassesAt = 16, kPartsAt = kPassesAt + 2 * kPassBytes;
static_assert(kKvMaxCtas * 4 % 16 == 0 && kPassBytes % 16 == 0 && kPartsAt % 16 == 0);

// At 256 channels the workspace has the former alone, and the tensor-core kernel as many CTAs as have their
// parts in it (94 of 152), or, for shared prefixes, the whole in the caller's scratch.
uint64_t few_bytes(int D) { return static_cast<uint64_t>(kKvMaxCtas) * 8 * (2 * (D + 2) + kWarps * D) * 4; }
uint64_t parts_bytes(int D) {
  const uint64_t few = few_bytes(D), many = D > 128 ? 0 : attention_block_bytes(D);
  return few > many ? few : many;
}
uint64_t scratch_parts_bytes(int D) { return D > 128 ? 2 * attention_block_bytes(D) : parts_bytes(D); }

void fill(AttnArgs& a, int D, const KvPool& pool, const KvBatch& kb, const void* q, int64_t q_stride, int heads, float scale, void* out,
          float* lse, void* workspace, int pass, void* parts) {
  a.pool = pool;
  a.kb = kb;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.heads = heads;
  a.group = heads / pool.kv_heads;
  a.scale_log2 = scale * 1.44269504088896f;
  a.window = 0;
  a.out = out;
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.err = reinterpret_cast<uint32_t*>(ws);
  uint8_t* own = ws + kPassesAt + pass * kPassBytes;
  a.counters = reinterpret_cast<uint32_t*>(own);
  a.joined = reinterpret_cast<Joined*>(own + kKvMaxCtas * 4);
  a.partial = static_cast<float*>(parts);
  a.stash = a.partial + static_cast<int64_t>(kKvMaxCtas) * 8 * 2 * (D + 2);
}

// Whether the tensor-core kernel takes `rows` query rows of `count` requests.
template <int SEE>
bool many_rows(int D, int64_t rows, int64_t count) { return (D <= 128 || SEE != kCausal) && rows >= kManyRows * count; }

// The CTAs whose parts (two each) have a place.
template <int SEE>
int most_block_ctas(int D, const AttnArgsOf<SEE>& a) {
  if constexpr (SEE != kCausal)
    if (D > 128 && a.pass == 0) return static_cast<int>(parts_bytes(D) / (attention_block_bytes(D) / (kKvMaxCtas / 2)));
  return kKvMaxCtas / 2;
}

template <int SEE>
cudaError_t launch_pass(int D, const AttnArgsOf<SEE>& a, int64_t count, int out_f32, const DeviceInfo& info, cudaStream_t s) {
  const int64_t rows = a.kb.tokens * a.group;
  if (many_rows<SEE>(D, rows, count)) return launch_attention_block<SEE>(D, a, count, most_block_ctas<SEE>(D, a), out_f32, info, s);
  return launch_attention_rows<SEE>(D, rows > 8 * count, a, out_f32, info, s);
}

}  // namespace

uint64_t attention_workspace_bytes(int D) { return kPartsAt + parts_bytes(D); }

uint64_t attention_shared_scratch(int D, int64_t tokens, int heads) {
  const uint64_t rows = static_cast<uint64_t>(tokens) * static_cast<uint64_t>(heads);
  return scratch_parts_bytes(D) + rows * static_cast<uint64_t>(D) * 4 + rows * 8;
}

cudaError_t launch_attention(int D, const KvPool& pool, const KvBatch& kb, const void* q, int64_t q_stride, int heads,
                             float scale, int64_t window, void* out, int out_f32, float* lse, void* workspace,
                             const DeviceInfo& info, cudaStream_t s) {
  AttnArgsOf<kCausal> a;
  fill(a, D, pool, kb, q, q_stride, heads, scale, out, lse, workspace, 0, static_cast<uint8_t*>(workspace) + kPartsAt);
  a.window = window > INT32_MAX ? 0 : window;          // positions have 31 bits: it hides nothing, and differences with it stay in 64
  return launch_pass<kCausal>(D, a, kb.batch, out_f32, info, s);
}

cudaError_t launch_attention_cross(int D, const KvPool& pool, const KvBatch& kb, const void* q, int64_t q_stride, int heads,
                                   float scale, void* out, int out_f32, float* lse, void* workspace, const DeviceInfo& info,
                                   cudaStream_t s) {
  AttnArgsOf<kAll> a;
  fill(a, D, pool, kb, q, q_stride, heads, scale, out, lse, workspace, 0, static_cast<uint8_t*>(workspace) + kPartsAt);
  return launch_pass<kAll>(D, a, kb.batch, out_f32, info, s);
}

cudaError_t launch_attention_shared(int D, const KvPool& pool, const KvBatch& kb, const int32_t* first, const int32_t* shared,
                                    int groups, const void* q, int64_t q_stride, int heads, float scale, void* out,
                                    int out_f32, float* lse, void* workspace, void* scratch, const DeviceInfo& info,
                                    cudaStream_t s) {
  AttnArgsOf<kAll> a;
  AttnArgsOf<kOwn> b;
  void* other = static_cast<uint8_t*>(D > 128 ? scratch : workspace) + (D > 128 ? attention_block_bytes(D) : kPartsAt);
  fill(a, D, pool, kb, q, q_stride, heads, scale, out, lse, workspace, 0, other);
  fill(b, D, pool, kb, q, q_stride, heads, scale, out, lse, workspace, 1, scratch);
  a.first = b.first = first;
  a.shared = b.shared = shared;
  a.groups = b.groups = groups;
  a.part_o = b.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + scratch_parts_bytes(D));
  a.part_ml = b.part_ml = reinterpret_cast<float2*>(a.part_o + kb.tokens * heads * D);
  // The tensor-core kernel has a second launch that joins its parts: it comes last, so
  // that nothing starts behind that launch.  Otherwise the prefixes, which are the larger part, come first
  // (16 requests behind 65537 positions: own parts first took 5 % more).  Both at the same time on SMs divided by what
  // they cost gained 3 of 60 us for 48 requests behind 8191 positions and took a model of the costs: not kept.
  const bool prefix_last = many_rows<kAll>(D, kb.tokens * a.group, groups) && !many_rows<kOwn>(D, kb.tokens * a.group, kb.batch);
  a.pass = prefix_last ? 2 : 1;
  b.pass = prefix_last ? 1 : 2;
  cudaError_t e = cudaSuccess;
  if (!prefix_last) e = launch_pass<kAll>(D, a, groups, out_f32, info, s);
  if (e == cudaSuccess) e = launch_pass<kOwn>(D, b, kb.batch, out_f32, info, s);
  if (e == cudaSuccess && prefix_last) e = launch_pass<kAll>(D, a, groups, out_f32, info, s);
  return e;
}

}  // namespace q4nx
