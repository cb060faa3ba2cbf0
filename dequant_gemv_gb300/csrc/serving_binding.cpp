// serving_binding.cpp -- the Python calls of the decode-step operators, as a
// CPython extension over the C ABI (include/q4nx.h).
//
// Like the ctypes binding it only marshals arguments: checks of types, shapes
// and devices, output tensors, the current stream, workspaces.  It is native
// because these calls are short: on one token the kernels take 5 to 10 us and the
// same checks and allocations in Python took 12 to 18 us a call.  A call here
// refuses what the Python binding refuses (ValueError), before anything runs; a status
// other than Q4NX_OK becomes the package's Q4NXError.  No C++ exception
// crosses into Python.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/q4nx.h"

namespace {

PyObject* g_error = nullptr;        // Q4NXError(status, where)
PyObject* g_workspace = nullptr;    // workspace(device, nbytes, family), makes or grows one
PyObject* g_workspaces = nullptr;   // the dictionary (family, device ordinal, stream) -> tensor

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};              // a Python exception is set already

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

// Refuse what is not a contiguous tensor of this type and number of dimensions on the call's device.
void plain(const at::Tensor& t, const char* name, at::ScalarType type, int64_t dims, c10::Device dev) {
  if (t.scalar_type() != type || t.dim() != dims || t.device() != dev || !t.is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of " + std::to_string(dims) +
                  " dimension(s) on " + dev.str());
}

void check(int status, const char* where) {
  if (status == Q4NX_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

struct Workspace {
  void* ptr;
  uint64_t bytes;
};
// The caller's workspace, or this stream's of the family.
Workspace workspace(PyObject* given, const char* family, c10::Device dev, cudaStream_t stream, uint64_t need) {
  if (given != Py_None) {
    const at::Tensor& t = tensor(given, "ws");
    if (!t.is_cuda() || !t.is_contiguous()) throw Refused("ws must be a contiguous CUDA tensor");
    return {t.data_ptr(), static_cast<uint64_t>(t.nbytes())};
  }
  PyObject* key = Py_BuildValue("siK", family, static_cast<int>(dev.index()), reinterpret_cast<unsigned long long>(stream));
  if (key == nullptr) throw PythonError();
  PyObject* have = PyDict_GetItemWithError(g_workspaces, key);      // borrowed; the dictionary keeps it
  Py_DECREF(key);
  if (have == nullptr && PyErr_Occurred()) throw PythonError();
  if (have != nullptr && static_cast<uint64_t>(THPVariable_Unpack(have).nbytes()) >= need)
    return {THPVariable_Unpack(have).data_ptr(), static_cast<uint64_t>(THPVariable_Unpack(have).nbytes())};
  PyObject* device = THPDevice_New(dev);
  PyObject* made = device ? PyObject_CallFunction(g_workspace, "OKs", device, static_cast<unsigned long long>(need), family) : nullptr;
  Py_XDECREF(device);
  if (made == nullptr) throw PythonError();
  const at::Tensor t = THPVariable_Unpack(made);
  Py_DECREF(made);                                                   // the dictionary keeps it
  return {t.data_ptr(), static_cast<uint64_t>(t.nbytes())};
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
at::ScalarType out_type(int64_t code) { return code == Q4NX_OUT_F32 ? at::kFloat : at::kBFloat16; }

q4nx_kv_batch batch_of(PyObject* const* args, int64_t tokens, c10::Device dev) {
  const at::Tensor &start = tensor(args[0], "q_start"), &lens = tensor(args[1], "lens"), &table = tensor(args[2], "table");
  plain(start, "q_start", at::kInt, 1, dev);
  plain(lens, "lens", at::kInt, 1, dev);
  plain(table, "table", at::kInt, 2, dev);
  const int64_t n = lens.numel();
  if (start.numel() != n + 1 || table.size(0) != n)
    throw Refused("q_start must have one entry more than lens, and table one row per request");
  if (n > INT32_MAX || table.size(1) > INT32_MAX) throw Refused("table is too large");
  q4nx_kv_batch b;
  b.q_start_dev = start.data_ptr<int32_t>();
  b.lens_dev = lens.data_ptr<int32_t>();
  b.table_dev = table.data_ptr<int32_t>();
  b.batch = static_cast<int32_t>(n);
  b.table_cols = static_cast<int32_t>(table.size(1));
  b.tokens = tokens;
  return b;
}

struct Rows {
  int64_t tokens, heads, stride;    // elements from token to token
};
// A bf16 [tokens, heads, head_dim] tensor with contiguous token rows.
Rows token_rows(const at::Tensor& t, const char* name, int64_t dim, c10::Device dev) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.device() != dev || t.size(2) != dim)
    throw Refused(std::string(name) + " must be a bf16 [tokens, heads, " + std::to_string(dim) + "] tensor on the cache's device");
  const int64_t n = t.size(0), heads = t.size(1);
  if (n > 0 && heads > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != dim)))
    throw Refused(std::string(name) + "'s heads must be contiguous within a token");
  return {n, heads, n > 1 ? t.stride(0) : heads * dim};
}

// ---- the calls; `cache` and `pool` come from a KVCache ----

struct Cache {
  const q4nx_kv_cache* c;
  c10::Device dev;
};
Cache cache_of(PyObject* address, PyObject* pool) {
  return {reinterpret_cast<const q4nx_kv_cache*>(static_cast<uintptr_t>(integer(address))), tensor(pool, "pool").device()};
}

// (cache, pool, ws_bytes, k, v, q_start, lens, table, ws)
PyObject* kv_append(PyObject* const* a) {
  const Cache cache = cache_of(a[0], a[1]);
  const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
  const Rows r = token_rows(k, "k", cache.c->head_dim, cache.dev), rv = token_rows(v, "v", cache.c->head_dim, cache.dev);
  if (r.tokens != rv.tokens || r.heads != rv.heads || r.stride != rv.stride || r.heads != cache.c->kv_heads)
    throw Refused("k and v must be [tokens, kv_heads, head_dim] with the same strides");
  const q4nx_kv_batch b = batch_of(a + 5, r.tokens, cache.dev);
  const c10::cuda::CUDAGuard guard(cache.dev);
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(cache.dev.index()).stream();
  const Workspace ws = workspace(a[8], "kv", cache.dev, s, static_cast<uint64_t>(integer(a[2])));
  if (r.tokens > 0)
    check(q4nx_kv_append(cache.c, &b, k.data_ptr(), v.data_ptr(), r.stride, ws.ptr, ws.bytes, s), "q4nx_kv_append");
  Py_RETURN_NONE;
}

// (cache, pool, ws_bytes, tokens, q_start, lens, table, out code, ws)
PyObject* kv_read(PyObject* const* a) {
  const Cache cache = cache_of(a[0], a[1]);
  const int64_t tokens = integer(a[3]), code = integer(a[7]);
  if (tokens < 0) throw Refused("tokens must not be negative");
  const q4nx_kv_batch b = batch_of(a + 4, tokens, cache.dev);
  const c10::cuda::CUDAGuard guard(cache.dev);
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(cache.dev.index()).stream();
  const Workspace ws = workspace(a[8], "kv", cache.dev, s, static_cast<uint64_t>(integer(a[2])));
  const int64_t shape[3] = {tokens, cache.c->kv_heads, cache.c->head_dim};
  at::Tensor k = empty(shape, out_type(code), cache.dev), v = empty(shape, out_type(code), cache.dev);
  if (tokens > 0)
    check(q4nx_kv_read(cache.c, &b, k.data_ptr(), v.data_ptr(), static_cast<int>(code), ws.ptr, ws.bytes, s), "q4nx_kv_read");
  return Py_BuildValue("NN", THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v)));
}

// (cache, pool, ws_bytes, q, q_start, lens, table, scale, window, out, out code, lse, ws)
PyObject* kv_attention(PyObject* const* a) {
  const Cache cache = cache_of(a[0], a[1]);
  const at::Tensor& q = tensor(a[3], "q");
  const Rows r = token_rows(q, "q", cache.c->head_dim, cache.dev);
  const q4nx_kv_batch b = batch_of(a + 4, r.tokens, cache.dev);
  const double scale = PyFloat_AsDouble(a[7]);
  if (scale == -1.0 && PyErr_Occurred()) throw PythonError();
  const int64_t window = integer(a[8]), code = integer(a[10]);
  const at::Tensor *given = tensor_or_none(a[9], "out"), *lse = tensor_or_none(a[11], "lse");
  const c10::cuda::CUDAGuard guard(cache.dev);
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(cache.dev.index()).stream();
  const Workspace ws = workspace(a[12], "kv", cache.dev, s, static_cast<uint64_t>(integer(a[2])));
  if (given != nullptr) {
    plain(*given, "out", out_type(code), 3, cache.dev);
    if (given->sizes() != q.sizes()) throw Refused("out must have q's shape");
  }
  if (lse != nullptr) {
    plain(*lse, "lse", at::kFloat, 2, cache.dev);
    if (lse->size(0) != r.tokens || lse->size(1) != r.heads) throw Refused("lse must be [tokens, heads]");
  }
  at::Tensor out = given != nullptr ? *given : empty(q.sizes(), out_type(code), cache.dev);
  if (r.tokens > 0)
    check(q4nx_kv_attention(cache.c, &b, q.data_ptr(), r.stride, static_cast<int>(r.heads), static_cast<float>(scale), window,
                            out.data_ptr(), static_cast<int>(code), lse != nullptr ? lse->data_ptr<float>() : nullptr, ws.ptr,
                            ws.bytes, s),
          "q4nx_kv_attention");
  return THPVariable_Wrap(std::move(out));
}

// (chunks, kind, rows, cols, X, adapters, their device ordinal, rows and cols, ids, out, out code, ws)
PyObject* gemm_lora(PyObject* const* a) {
  const at::Tensor &chunks = tensor(a[0], "chunks"), &x = tensor(a[4], "X"), &ids = tensor(a[9], "ids");
  if (!chunks.is_cuda() || !chunks.is_contiguous()) throw Refused("chunks must be a contiguous CUDA tensor");
  const c10::Device dev = chunks.device();
  q4nx_weight w;
  w.chunks_dev = chunks.data_ptr();
  w.bytes = static_cast<uint64_t>(chunks.nbytes());
  w.kind = static_cast<int32_t>(integer(a[1]));
  w.reserved = 0;
  w.rows = integer(a[2]);
  w.cols = integer(a[3]);
  const q4nx_adapters* ad = reinterpret_cast<const q4nx_adapters*>(static_cast<uintptr_t>(integer(a[5])));
  plain(x, "X", at::kBFloat16, 2, dev);
  plain(ids, "ids", at::kInt, 1, dev);
  const int64_t M = x.size(0), code = integer(a[11]);
  if (x.size(1) != w.cols || integer(a[6]) != dev.index() || integer(a[7]) != w.rows || integer(a[8]) != w.cols)
    throw Refused("X must be [M, cols], and the adapters the weight's: a [count, rank, cols], b [count, rows, rank]");
  if (ids.numel() != M) throw Refused("ids must have one entry per token");
  const at::Tensor* given = tensor_or_none(a[10], "out");
  const int m = static_cast<int>(M < INT32_MAX ? M : INT32_MAX);
  if (m < 1 || m > 64) check(Q4NX_E_M, "q4nx_gemm_lora");
  const int64_t shape[2] = {M, w.rows};
  if (given != nullptr) {
    plain(*given, "out", out_type(code), 2, dev);
    if (given->size(0) != M || given->size(1) != w.rows) throw Refused("out must be [M, rows]");
  }
  const uint64_t need = q4nx_gemm_workspace(&w, m);
  if (need == 0) check(Q4NX_E_SHAPE, "q4nx_gemm_lora");
  const c10::cuda::CUDAGuard guard(dev);
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const Workspace ws = workspace(a[12], "gemm", dev, s, need);
  at::Tensor out = given != nullptr ? *given : empty(shape, out_type(code), dev);
  // scratch of any content: the caching allocator keeps it to this stream's order
  const int64_t bytes = static_cast<int64_t>(q4nx_gemm_lora_scratch(&w, m));
  const at::Tensor scratch = empty(bytes, at::kByte, dev);
  check(q4nx_gemm_lora(&w, x.data_ptr(), m, ad, ids.data_ptr<int32_t>(), out.data_ptr(), static_cast<int>(code), ws.ptr, ws.bytes,
                       scratch.data_ptr(), static_cast<uint64_t>(bytes), s),
        "q4nx_gemm_lora");
  return THPVariable_Wrap(std::move(out));
}

// (logits, tokens, top) -> (logprob, entropy, lse, top_idx, top_logprob)
PyObject* logprobs(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const at::Tensor* tokens = tensor_or_none(a[1], "tokens");
  const int64_t top = integer(a[2]);
  if (!x.is_cuda() || x.dim() != 2 || (x.scalar_type() != at::kFloat && x.scalar_type() != at::kBFloat16))
    throw Refused("logits must be a CUDA tensor, fp32 or bf16 [M, V]");
  const c10::Device dev = x.device();
  const int64_t M = x.size(0), V = x.size(1);
  if (V > 1 && x.stride(1) != 1) throw Refused("a row of logits must be contiguous");
  if (top < 0 || top > Q4NX_MAX_TOP) throw Refused("top must be in 0.." + std::to_string(Q4NX_MAX_TOP));
  if (M > 65535) check(Q4NX_E_SHAPE, "q4nx_logprobs");
  if (tokens != nullptr) {
    plain(*tokens, "tokens", at::kInt, 1, dev);
    if (tokens->numel() != M) throw Refused("tokens must have one entry per row");
  }
  const c10::cuda::CUDAGuard guard(dev);
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const int64_t pair[2] = {M, top};
  at::Tensor lp, entropy = empty(M, at::kFloat, dev), lse = empty(M, at::kFloat, dev), idx = empty(pair, at::kInt, dev),
                 tlp = empty(pair, at::kFloat, dev);
  if (tokens != nullptr) lp = empty(M, at::kFloat, dev);
  check(q4nx_logprobs(x.data_ptr(), x.scalar_type() == at::kFloat ? Q4NX_OUT_F32 : Q4NX_OUT_BF16, static_cast<int>(M), V,
                      M > 1 ? x.stride(0) : V, tokens != nullptr ? tokens->data_ptr<int32_t>() : nullptr, static_cast<int>(top),
                      tokens != nullptr ? lp.data_ptr<float>() : nullptr, entropy.data_ptr<float>(), lse.data_ptr<float>(),
                      idx.data_ptr<int32_t>(), tlp.data_ptr<float>(), s),
        "q4nx_logprobs");
  PyObject* first = tokens != nullptr ? THPVariable_Wrap(std::move(lp)) : Py_NewRef(Py_None);
  return Py_BuildValue("NNNNN", first, THPVariable_Wrap(std::move(entropy)), THPVariable_Wrap(std::move(lse)),
                       THPVariable_Wrap(std::move(idx)), THPVariable_Wrap(std::move(tlp)));
}

// A call with its number of arguments checked and its exceptions turned into Python's.
template <PyObject* (*Call)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, not %zd", N, n);
    return nullptr;
  }
  try {
    return Call(args);
  } catch (const PythonError&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (error class, workspace function, workspace dictionary)
PyObject* setup(PyObject* const* a) {
  for (int i = 0; i < 3; ++i) Py_INCREF(a[i]);
  g_error = a[0];
  g_workspace = a[1];
  g_workspaces = a[2];
  Py_RETURN_NONE;
}

template <PyObject* (*Call)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<Call, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<setup, 3>("setup"),
                           method<kv_append, 9>("kv_append"),
                           method<kv_read, 9>("kv_read"),
                           method<kv_attention, 13>("kv_attention"),
                           method<gemm_lora, 13>("gemm_lora"),
                           method<logprobs, 3>("logprobs"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&g_module); }
