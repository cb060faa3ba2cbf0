"""The operators around the products in a decode step, as Python calls.

    KVCache.alloc(pages, kv_heads, head_dim, page_tokens, device)
    q4nx_kv_append(cache, k, v, q_start, lens, table)
    q4nx_kv_append_rotary(cache, Rotary(table), q, k, v, q_start, lens, table) -> turned q
    q4nx_kv_read(cache, tokens, q_start, lens, table)            -> (k, v)
    q4nx_kv_attention(cache, q, q_start, lens, table, scale)     -> [tokens, heads, head_dim]
    q4nx_kv_attention_cross(cache, q, q_start, lens, table, scale)                  -> [tokens, heads, head_dim]
    q4nx_kv_attention_shared(cache, q, q_start, lens, table, first, shared, scale)  -> [tokens, heads, head_dim]
    q4nx_gemm_lora(w, X, Adapters(a, b, scale), ids)             -> [M, N]
    q4nx_gemm_epilogue(w, X, bias, act, mul, residual)           -> [M, N]
    q4nx_logprobs(logits, tokens, top)                           -> Logprobs

As in the rest of the binding, only arguments are marshalled; formulas,
layouts and limits stand in ``include/q4nx.h``.  The marshalling itself is native
(``csrc/serving_binding.cpp``): it is as long as the kernels of small calls.  Where
that binding has not been built these calls raise ImportError; the products need none of it.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import Q4NXError, Weight, _out_code, _ws, lib, q4nx_weight, workspace


class _NotBuilt:
    """In the place of the binding: every call of it says why there is none."""

    def __init__(self, why: ImportError):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name}: the native binding _serving.so is not usable ({self._why}); "
                          "build it with python dequant_gemv_gb300/_build.py") from self._why


try:
    from . import _serving
except ImportError as e:                 # not built, or built for another torch or Python
    _serving = _NotBuilt(e)
else:
    _serving.setup(Q4NXError, workspace, _ws)
P, U64, I, I64, F = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class q4nx_kv_cache(ctypes.Structure):
    _fields_ = [("pool_dev", P), ("bytes", U64), ("head_dim", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32), ("pages", I64)]


class q4nx_kv_batch(ctypes.Structure):
    _fields_ = [("q_start_dev", P), ("lens_dev", P), ("table_dev", P), ("batch", ctypes.c_int32),
                ("table_cols", ctypes.c_int32), ("tokens", I64)]


class q4nx_kv_groups(ctypes.Structure):
    _fields_ = [("first_dev", P), ("shared_dev", P), ("count", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class q4nx_adapters(ctypes.Structure):
    _fields_ = [("a_dev", P), ("b_dev", P), ("scale_dev", P), ("a_bytes", U64), ("b_bytes", U64),
                ("count", ctypes.c_int32), ("rank", ctypes.c_int32)]


class q4nx_rotary(ctypes.Structure):
    _fields_ = [("table_dev", P), ("bytes", U64), ("positions", I64), ("dims", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class q4nx_epilogue(ctypes.Structure):
    _fields_ = [("bias_dev", P), ("mul_dev", P), ("residual_dev", P), ("mul_stride", I64), ("residual_stride", I64),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_CACHE, _BATCH = ctypes.POINTER(q4nx_kv_cache), ctypes.POINTER(q4nx_kv_batch)
for _name, (_args, _res) in {
    "q4nx_kv_page_bytes": ([I, I, I], U64),
    "q4nx_kv_workspace": ([_CACHE], U64),
    "q4nx_kv_append": ([_CACHE, _BATCH, P, P, I64, P, U64, P], I),
    "q4nx_kv_append_rotary": ([_CACHE, _BATCH, ctypes.POINTER(q4nx_rotary), P, I64, I, P, I64, P, P, I64, P, U64, P], I),
    "q4nx_kv_read": ([_CACHE, _BATCH, P, P, I, P, U64, P], I),
    "q4nx_kv_attention": ([_CACHE, _BATCH, P, I64, I, F, I64, P, I, P, P, U64, P], I),
    "q4nx_kv_attention_cross": ([_CACHE, _BATCH, P, I64, I, F, P, I, P, P, U64, P], I),
    "q4nx_kv_attention_shared": ([_CACHE, _BATCH, ctypes.POINTER(q4nx_kv_groups), P, I64, I, F, P, I, P, P, U64, P, U64, P], I),
    "q4nx_kv_attention_shared_scratch": ([_CACHE, I64, I], U64),
    "q4nx_gemm_lora": ([ctypes.POINTER(q4nx_weight), P, I, ctypes.POINTER(q4nx_adapters), P, P, I, P, U64, P, U64, P], I),
    "q4nx_gemm_lora_scratch": ([ctypes.POINTER(q4nx_weight), I], U64),
    "q4nx_gemm_epilogue": ([ctypes.POINTER(q4nx_weight), P, I, ctypes.POINTER(q4nx_epilogue), P, I, P, U64, P], I),
    "q4nx_logprobs": ([P, I, I, I64, I64, P, I, P, P, P, P, P, P], I),
}.items():
    _fn = getattr(lib, _name)
    _fn.argtypes, _fn.restype = _args, _res
EXPORTS = ("q4nx_kv_page_bytes", "q4nx_kv_workspace", "q4nx_kv_append", "q4nx_kv_append_rotary", "q4nx_kv_read", "q4nx_kv_attention",
           "q4nx_kv_attention_cross", "q4nx_kv_attention_shared", "q4nx_kv_attention_shared_scratch",
           "q4nx_gemm_lora", "q4nx_gemm_lora_scratch", "q4nx_gemm_epilogue", "q4nx_logprobs")
Q4NX_MAX_TOP = 32
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}       # enum q4nx_act


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
        object.__setattr__(self, "_at", ctypes.addressof(c))
        object.__setattr__(self, "_ws_bytes", int(lib.q4nx_kv_workspace(ctypes.byref(c))))

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


def q4nx_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor,
                   table: torch.Tensor, ws: torch.Tensor | None = None) -> None:
    """Quantize new keys and values (bf16 [tokens, kv_heads, head_dim]) into the cache; lens counts them already."""
    _serving.kv_append(cache._at, cache.pool, cache._ws_bytes, k, v, q_start, lens, table, ws)


@dataclass(frozen=True)
class Rotary:
    """Cosines and sines of the positions: fp32 [positions, dims / 2, 2].

    The first dims channels of a head are turned, in pairs (j, j + dims / 2), or (2j, 2j + 1) where interleaved."""
    table: torch.Tensor
    interleaved: bool = False

    def __post_init__(self):
        t = self.table
        if t.dtype != torch.float32 or t.dim() != 3 or t.shape[2] != 2 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("table must be a contiguous fp32 CUDA tensor [positions, dims / 2, 2]")
        c = q4nx_rotary(t.data_ptr(), t.numel() * 4, t.shape[0], 2 * t.shape[1], int(bool(self.interleaved)))
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_at", ctypes.addressof(c))

    @classmethod
    def make(cls, positions: int, dims: int, base: float = 10000.0, frequencies: torch.Tensor | None = None,
             interleaved: bool = False, device="cuda") -> "Rotary":
        """The table of angles position * frequencies[j] (base ** (-2j / dims) by default), computed in 64 bits."""
        if frequencies is None:
            frequencies = base ** (-2 * torch.arange(dims // 2, dtype=torch.float64, device=device) / dims)
        if frequencies.shape != (dims // 2,):
            raise ValueError("frequencies must be [dims / 2]")
        angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * frequencies.to(device=device, dtype=torch.float64)
        return cls(torch.stack([angle.cos(), angle.sin()], -1).float(), interleaved)

    def c(self) -> q4nx_rotary:
        return self._c


def q4nx_kv_append_rotary(cache: KVCache, rotary: Rotary, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor,
                          lens: torch.Tensor, table: torch.Tensor, out: torch.Tensor | None = None,
                          ws: torch.Tensor | None = None) -> torch.Tensor | None:
    """q4nx_kv_append with keys and queries (bf16 [tokens, heads, head_dim], or None) turned by their positions; the turned queries.

    out: their place (it may be q)."""
    return _serving.kv_append_rotary(cache._at, cache.pool, cache._ws_bytes, rotary._at, rotary.table, q, k, v, q_start, lens, table, out, ws)


def q4nx_kv_read(cache: KVCache, tokens: int, q_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                 out_dtype="bf16", ws: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The cached values of the last q_start[b+1] - q_start[b] tokens of every request, [tokens, kv_heads, head_dim] each."""
    return _serving.kv_read(cache._at, cache.pool, cache._ws_bytes, tokens, q_start, lens, table, _out_code(out_dtype), ws)


def q4nx_kv_attention(cache: KVCache, q: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                      scale: float | None = None, window: int = 0, out: torch.Tensor | None = None, out_dtype="bf16",
                      lse: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the requests' newest tokens over their caches.

    q: bf16 [tokens, heads, head_dim]; scale: 1/sqrt(head_dim) by default;
    window: 0 for none; lse: fp32 [tokens, heads] to be filled, or None."""
    return _serving.kv_attention(cache._at, cache.pool, cache._ws_bytes, q, q_start, lens, table,
                                 cache.head_dim ** -0.5 if scale is None else scale, window, out, _out_code(out_dtype), lse, ws)


def q4nx_kv_attention_cross(cache: KVCache, q: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                            scale: float | None = None, out: torch.Tensor | None = None, out_dtype="bf16",
                            lse: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the requests' tokens to all positions of another sequence's cache; lens: its lengths.

    Other arguments as of q4nx_kv_attention."""
    return _serving.kv_attention_cross(cache._at, cache.pool, cache._ws_bytes, q, q_start, lens, table,
                                       cache.head_dim ** -0.5 if scale is None else scale, out, _out_code(out_dtype), lse, ws)


def q4nx_kv_attention_shared(cache: KVCache, q: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                             first: torch.Tensor, shared: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
                             out_dtype="bf16", lse: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """q4nx_kv_attention of requests that share prefixes, each read once.

    first: int32 [groups + 1], the groups' first requests and the batch; shared: int32 [groups], the
    positions that a group's requests have in common (lens counts them); other arguments as of q4nx_kv_attention."""
    return _serving.kv_attention_shared(cache._at, cache.pool, cache._ws_bytes, q, q_start, lens, table,
                                        cache.head_dim ** -0.5 if scale is None else scale, first, shared, out, _out_code(out_dtype), lse, ws)


@dataclass(frozen=True)
class Adapters:
    """Low-rank adapters of one projection: a bf16 [count, rank, cols], b bf16 [count, rows, rank], scale fp32 [count]."""
    a: torch.Tensor
    b: torch.Tensor
    scale: torch.Tensor

    def __post_init__(self):
        a, b, scale = self.a, self.b, self.scale
        for t, dtype, dims in ((a, torch.bfloat16, 3), (b, torch.bfloat16, 3), (scale, torch.float32, 1)):
            if t.dtype != dtype or t.dim() != dims or not t.is_cuda or t.device != a.device or not t.is_contiguous():
                raise ValueError("adapters must be contiguous CUDA tensors: a, b bf16 of 3 dimensions, scale fp32 of one")
        n, rank, cols = a.shape
        if b.shape[0] != n or b.shape[2] != rank or scale.numel() != n:
            raise ValueError("adapters must be a [count, rank, cols], b [count, rows, rank], scale [count]")
        c = q4nx_adapters(a.data_ptr(), b.data_ptr(), scale.data_ptr(), a.numel() * 2, b.numel() * 2, n, rank)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_fits", (ctypes.addressof(c), a.device.index, b.shape[1], cols))

    def c(self) -> q4nx_adapters:
        return self._c


def q4nx_gemm_lora(w: Weight, X: torch.Tensor, adapters: Adapters, ids: torch.Tensor, out: torch.Tensor | None = None,
                   out_dtype="bf16", ws: torch.Tensor | None = None) -> torch.Tensor:
    """w X[m] plus the adapter ids[m] (int32, below 0: none) of every token, [M, rows]."""
    return _serving.gemm_lora(w.chunks, w.kind, w.rows, w.cols, X, *adapters._fits, ids, out, _out_code(out_dtype), ws)


def q4nx_gemm_epilogue(w: Weight, X: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none", mul: torch.Tensor | None = None,
                       residual: torch.Tensor | None = None, out: torch.Tensor | None = None, out_dtype="bf16",
                       ws: torch.Tensor | None = None) -> torch.Tensor:
    """act(w X[m] + bias) * mul[m] + residual[m], [M, rows]; bias bf16 [rows], mul and residual bf16 [M, rows].

    act: one of ACTIVATIONS; out may be mul or residual (a contiguous bf16 one)."""
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}")
    return _serving.gemm_epilogue(w.chunks, w.kind, w.rows, w.cols, X, bias, ACTIVATIONS[act], mul, residual, out, _out_code(out_dtype), ws)


class Logprobs(NamedTuple):
    logprob: torch.Tensor | None      # fp32 [M], the given tokens'
    entropy: torch.Tensor             # fp32 [M]
    lse: torch.Tensor                 # fp32 [M]
    top_idx: torch.Tensor             # int32 [M, top], largest first
    top_logprob: torch.Tensor         # fp32 [M, top]


def q4nx_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0) -> Logprobs:
    """Log-probability of each row's token (int32 [M]), entropy and the `top` most likely tokens of logits [M, V]."""
    return Logprobs(*_serving.logprobs(logits, tokens, top))
