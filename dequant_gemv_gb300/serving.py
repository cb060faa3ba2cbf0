"""The operators around the products in a decode step, as Python calls.

    KVCache.alloc(pages, kv_heads, head_dim, page_tokens, device)
    q4nx_kv_append(cache, k, v, q_start, lens, table)
    q4nx_kv_read(cache, tokens, q_start, lens, table)            -> (k, v)
    q4nx_kv_attention(cache, q, q_start, lens, table, scale)     -> [tokens, heads, head_dim]
    q4nx_gemm_lora(w, X, Adapters(a, b, scale), ids)             -> [M, N]
    q4nx_logprobs(logits, tokens, top)                           -> Logprobs

As in the rest of the binding, only arguments are marshalled here; formulas,
layouts and limits stand in ``include/q4nx.h``.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import Weight, _check, _out_code, _ws, lib, q4nx_weight, workspace

# the current device's ordinal, and the handle of its current stream, without a Stream object (2 us a call)
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_byref = ctypes.byref
P, U64, I, I64, F = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class q4nx_kv_cache(ctypes.Structure):
    _fields_ = [("pool_dev", P), ("bytes", U64), ("head_dim", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32), ("pages", I64)]


class q4nx_kv_batch(ctypes.Structure):
    _fields_ = [("q_start_dev", P), ("lens_dev", P), ("table_dev", P), ("batch", ctypes.c_int32),
                ("table_cols", ctypes.c_int32), ("tokens", I64)]


class q4nx_adapters(ctypes.Structure):
    _fields_ = [("a_dev", P), ("b_dev", P), ("scale_dev", P), ("a_bytes", U64), ("b_bytes", U64),
                ("count", ctypes.c_int32), ("rank", ctypes.c_int32)]


_CACHE, _BATCH = ctypes.POINTER(q4nx_kv_cache), ctypes.POINTER(q4nx_kv_batch)
for _name, (_args, _res) in {
    "q4nx_kv_page_bytes": ([I, I, I], U64),
    "q4nx_kv_workspace": ([_CACHE], U64),
    "q4nx_kv_append": ([_CACHE, _BATCH, P, P, I64, P, U64, P], I),
    "q4nx_kv_read": ([_CACHE, _BATCH, P, P, I, P, U64, P], I),
    "q4nx_kv_attention": ([_CACHE, _BATCH, P, I64, I, F, I64, P, I, P, P, U64, P], I),
    "q4nx_gemm_lora": ([ctypes.POINTER(q4nx_weight), P, I, ctypes.POINTER(q4nx_adapters), P, P, I, P, U64, P, U64, P], I),
    "q4nx_gemm_lora_scratch": ([ctypes.POINTER(q4nx_weight), I], U64),
    "q4nx_logprobs": ([P, I, I, I64, I64, P, I, P, P, P, P, P, P], I),
}.items():
    _fn = getattr(lib, _name)
    _fn.argtypes, _fn.restype = _args, _res
EXPORTS = ("q4nx_kv_page_bytes", "q4nx_kv_workspace", "q4nx_kv_append", "q4nx_kv_read", "q4nx_kv_attention",
           "q4nx_gemm_lora", "q4nx_gemm_lora_scratch", "q4nx_logprobs")
Q4NX_MAX_TOP = 32


def q4nx_kv_page_bytes(head_dim: int, kv_heads: int, page_tokens: int) -> int:
    return int(lib.q4nx_kv_page_bytes(head_dim, kv_heads, page_tokens))


@dataclass(frozen=True)
class KVCache:
    """A pool of pages (uint8 CUDA tensor) that hold keys and values in 4 bits."""
    pool: torch.Tensor
    head_dim: int
    kv_heads: int
    page_tokens: int
    pages: int

    def __post_init__(self):
        if not self.pool.is_cuda or not self.pool.is_contiguous():
            raise ValueError("pool must be a contiguous CUDA tensor")
        c = q4nx_kv_cache(self.pool.data_ptr(), self.pool.numel() * self.pool.element_size(), int(self.head_dim),
                          int(self.kv_heads), int(self.page_tokens), 0, int(self.pages))
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ws_bytes", int(lib.q4nx_kv_workspace(_byref(c))))

    @classmethod
    def alloc(cls, pages: int, kv_heads: int, head_dim: int, page_tokens: int, device="cuda") -> "KVCache":
        page = q4nx_kv_page_bytes(head_dim, kv_heads, page_tokens)
        if page == 0 or pages < 1:
            raise ValueError("head_dim must be 64, 128 or 256, page_tokens a positive multiple of 16, kv_heads and pages positive")
        return cls(torch.empty(pages * page, dtype=torch.uint8, device=device), head_dim, kv_heads, page_tokens, pages)

    def c(self) -> q4nx_kv_cache:
        return self._c

    @property
    def device(self) -> torch.device:
        return self.pool.device


def _plain(t: torch.Tensor, name: str, dtype: torch.dtype, dims: int, dev: torch.device) -> None:
    """Refuse what is not a contiguous tensor of this type and number of dimensions on the call's device."""
    if t.dtype is not dtype or t.dim() != dims or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {dims} dimension(s) on {dev}")


def _workspace(dev: torch.device, stream: int, nbytes: int, family: str) -> torch.Tensor:
    ws = _ws.get((family, dev.index, stream))
    return ws if ws is not None and ws.numel() >= nbytes else workspace(dev, nbytes, family)


def _batch(dev: torch.device, tokens: int, q_start, lens, table) -> q4nx_kv_batch:
    _plain(q_start, "q_start", torch.int32, 1, dev)
    _plain(lens, "lens", torch.int32, 1, dev)
    _plain(table, "table", torch.int32, 2, dev)
    n, (rows, cols) = lens.numel(), table.shape
    if q_start.numel() != n + 1 or rows != n:
        raise ValueError("q_start must have one entry more than lens, and table one row per request")
    return q4nx_kv_batch(q_start.data_ptr(), lens.data_ptr(), table.data_ptr(), n, cols, tokens)


def _token_rows(t: torch.Tensor, name: str, cache: KVCache) -> tuple[int, int, int]:
    """(tokens, heads, elements from token to token) of a bf16 [tokens, heads, head_dim] tensor with contiguous token rows."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.device != cache.pool.device:
        raise ValueError(f"{name} must be a bf16 [tokens, heads, {cache.head_dim}] tensor on the cache's device")
    (n, heads, d), (s0, s1, s2) = t.shape, t.stride()
    if d != cache.head_dim:
        raise ValueError(f"{name} must have {cache.head_dim} channels per head")
    if n and heads and (s2 != 1 or (heads > 1 and s1 != d)):
        raise ValueError(f"{name}'s heads must be contiguous within a token")
    return n, heads, s0 if n > 1 else heads * d


def q4nx_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor,
                   table: torch.Tensor, ws: torch.Tensor | None = None) -> None:
    """Quantize new keys and values (bf16 [tokens, kv_heads, head_dim]) into the cache; lens counts them already."""
    dev = cache.pool.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return q4nx_kv_append(cache, k, v, q_start, lens, table, ws)
    rows = _token_rows(k, "k", cache)
    if rows != _token_rows(v, "v", cache) or rows[1] != cache.kv_heads:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] with the same strides")
    cb, stream = _batch(dev, rows[0], q_start, lens, table), _raw_stream(dev.index)
    if ws is None:
        ws = _workspace(dev, stream, cache._ws_bytes, "kv")
    if rows[0]:
        _check(lib.q4nx_kv_append(_byref(cache._c), _byref(cb), k.data_ptr(), v.data_ptr(), rows[2], ws.data_ptr(),
                                  ws.numel(), stream), "q4nx_kv_append")


def q4nx_kv_read(cache: KVCache, tokens: int, q_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                 out_dtype="bf16", ws: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The cached values of the last q_start[b+1] - q_start[b] tokens of every request, [tokens, kv_heads, head_dim] each."""
    dev = cache.pool.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return q4nx_kv_read(cache, tokens, q_start, lens, table, out_dtype, ws)
    cb, code, stream = _batch(dev, tokens, q_start, lens, table), _out_code(out_dtype), _raw_stream(dev.index)
    if ws is None:
        ws = _workspace(dev, stream, cache._ws_bytes, "kv")
    shape, dt = (tokens, cache.kv_heads, cache.head_dim), torch.float32 if code else torch.bfloat16
    k, v = torch.empty(shape, dtype=dt, device=dev), torch.empty(shape, dtype=dt, device=dev)
    if tokens:
        _check(lib.q4nx_kv_read(_byref(cache._c), _byref(cb), k.data_ptr(), v.data_ptr(), code, ws.data_ptr(),
                                ws.numel(), stream), "q4nx_kv_read")
    return k, v


def q4nx_kv_attention(cache: KVCache, q: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                      scale: float | None = None, window: int = 0, out: torch.Tensor | None = None, out_dtype="bf16",
                      lse: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the requests' newest tokens over their caches.

    q: bf16 [tokens, heads, head_dim]; scale: 1/sqrt(head_dim) by default;
    window: 0 for none; lse: fp32 [tokens, heads] to be filled, or None."""
    dev = cache.pool.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return q4nx_kv_attention(cache, q, q_start, lens, table, scale, window, out, out_dtype, lse, ws)
    tokens, heads, stride = _token_rows(q, "q", cache)
    cb, code, stream = _batch(dev, tokens, q_start, lens, table), _out_code(out_dtype), _raw_stream(dev.index)
    if ws is None:
        ws = _workspace(dev, stream, cache._ws_bytes, "kv")
    dt = torch.float32 if code else torch.bfloat16
    if out is None:
        out = torch.empty((tokens, heads, cache.head_dim), dtype=dt, device=dev)
    else:
        _plain(out, "out", dt, 3, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    lse_ptr = None
    if lse is not None:
        _plain(lse, "lse", torch.float32, 2, dev)
        if lse.shape != (tokens, heads):
            raise ValueError("lse must be [tokens, heads]")
        lse_ptr = lse.data_ptr()
    if tokens:
        _check(lib.q4nx_kv_attention(_byref(cache._c), _byref(cb), q.data_ptr(), stride, heads,
                                     cache.head_dim ** -0.5 if scale is None else scale, window, out.data_ptr(), code,
                                     lse_ptr, ws.data_ptr(), ws.numel(), stream), "q4nx_kv_attention")
    return out


@dataclass(frozen=True)
class Adapters:
    """Low-rank adapters of one projection: a bf16 [count, rank, cols], b bf16 [count, rows, rank], scale fp32 [count]."""
    a: torch.Tensor
    b: torch.Tensor
    scale: torch.Tensor

    def __post_init__(self):
        dev = self.a.device
        _plain(self.a, "a", torch.bfloat16, 3, dev)
        _plain(self.b, "b", torch.bfloat16, 3, dev)
        _plain(self.scale, "scale", torch.float32, 1, dev)
        n, rank, _ = self.a.shape
        if self.b.shape[0] != n or self.b.shape[2] != rank or self.scale.numel() != n or dev.type != "cuda":
            raise ValueError("adapters must be CUDA tensors a [count, rank, cols], b [count, rows, rank], scale [count]")
        object.__setattr__(self, "_c", q4nx_adapters(self.a.data_ptr(), self.b.data_ptr(), self.scale.data_ptr(),
                                                     self.a.numel() * 2, self.b.numel() * 2, n, rank))
        object.__setattr__(self, "_fits", (dev, self.b.shape[1], self.a.shape[2]))

    def c(self) -> q4nx_adapters:
        return self._c


def q4nx_gemm_lora(w: Weight, X: torch.Tensor, adapters: Adapters, ids: torch.Tensor, out: torch.Tensor | None = None,
                   out_dtype="bf16", ws: torch.Tensor | None = None) -> torch.Tensor:
    """w X[m] plus the adapter ids[m] (int32, below 0: none) of every token, [M, rows]."""
    dev = w.chunks.device
    if not w.chunks.is_cuda or not w.chunks.is_contiguous():
        raise ValueError("chunks must be a contiguous CUDA tensor")
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return q4nx_gemm_lora(w, X, adapters, ids, out, out_dtype, ws)
    _plain(X, "X", torch.bfloat16, 2, dev)
    _plain(ids, "ids", torch.int32, 1, dev)
    M, cols = X.shape
    if cols != w.cols or adapters._fits != (dev, w.rows, w.cols):
        raise ValueError("X must be [M, cols], and the adapters the weight's: a [count, rank, cols], b [count, rows, rank]")
    if ids.numel() != M:
        raise ValueError("ids must have one entry per token")
    code, stream, cw = _out_code(out_dtype), _raw_stream(dev.index), w.c()
    dt = torch.float32 if code else torch.bfloat16
    if out is None:
        out = torch.empty((M, w.rows), dtype=dt, device=dev)
    else:
        _plain(out, "out", dt, 2, dev)
        if out.shape != (M, w.rows):
            raise ValueError("out must be [M, rows]")
    if ws is None:
        ws = _workspace(dev, stream, int(lib.q4nx_gemm_workspace(_byref(cw), M)), "gemm")
    # scratch of any content: the caching allocator keeps it to this stream's order
    scratch = torch.empty(lib.q4nx_gemm_lora_scratch(_byref(cw), M), dtype=torch.uint8, device=dev)
    _check(lib.q4nx_gemm_lora(_byref(cw), X.data_ptr(), M, _byref(adapters._c), ids.data_ptr(), out.data_ptr(), code,
                              ws.data_ptr(), ws.numel(), scratch.data_ptr(), scratch.numel(), stream), "q4nx_gemm_lora")
    return out


class Logprobs(NamedTuple):
    logprob: torch.Tensor | None      # fp32 [M], the given tokens'
    entropy: torch.Tensor             # fp32 [M]
    lse: torch.Tensor                 # fp32 [M]
    top_idx: torch.Tensor             # int32 [M, top], largest first
    top_logprob: torch.Tensor         # fp32 [M, top]


def q4nx_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0) -> Logprobs:
    """Log-probability of each row's token (int32 [M]), entropy and the `top` most likely tokens of logits [M, V]."""
    dev = logits.device
    if not logits.is_cuda or logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be a CUDA tensor, fp32 or bf16 [M, V]")
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return q4nx_logprobs(logits, tokens, top)
    (M, V), (pitch, step) = logits.shape, logits.stride()
    if V > 1 and step != 1:
        raise ValueError("a row of logits must be contiguous")
    if not 0 <= top <= Q4NX_MAX_TOP:
        raise ValueError(f"top must be in 0..{Q4NX_MAX_TOP}")
    lp = lp_ptr = tok_ptr = None
    if tokens is not None:
        _plain(tokens, "tokens", torch.int32, 1, dev)
        if tokens.numel() != M:
            raise ValueError("tokens must have one entry per row")
        lp = torch.empty(M, dtype=torch.float32, device=dev)
        lp_ptr, tok_ptr = lp.data_ptr(), tokens.data_ptr()
    ent, lse = torch.empty(M, dtype=torch.float32, device=dev), torch.empty(M, dtype=torch.float32, device=dev)
    idx, tlp = torch.empty((M, top), dtype=torch.int32, device=dev), torch.empty((M, top), dtype=torch.float32, device=dev)
    _check(lib.q4nx_logprobs(logits.data_ptr(), 1 if logits.dtype is torch.float32 else 0, M, V, pitch if M > 1 else V,
                             tok_ptr, top, lp_ptr, ent.data_ptr(), lse.data_ptr(), idx.data_ptr(), tlp.data_ptr(),
                             _raw_stream(dev.index)), "q4nx_logprobs")
    return Logprobs(lp, ent, lse, idx, tlp)
