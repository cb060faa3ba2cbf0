"""Host-side checks of the decode-step operators (no GPU needed): sizes, and the
documented status for every bad argument, before any CUDA call."""
import ctypes

import pytest
import torch

P = 0x10000                      # a fake, aligned "device" address: never dereferenced


@pytest.fixture(scope="module")
def q():
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    import dequant_gemv_gb300

    return dequant_gemv_gb300


def _cache(q, pool=P, nbytes=1 << 30, dim=128, heads=8, page=64, reserved=0, pages=10):
    return q.q4nx_kv_cache(pool, nbytes, dim, heads, page, reserved, pages)


def _batch(q, a=P, b=P, c=P, batch=3, cols=4, tokens=3):
    return q.q4nx_kv_batch(a, b, c, batch, cols, tokens)


def test_page_bytes(q):
    # 4-bit codes, and a bf16 scale and middle per 32 channels, of keys and values
    for dim in (64, 128, 256):
        assert q.q4nx_kv_page_bytes(dim, 3, 48) == 48 * 3 * 2 * (dim // 2 + dim // 32 * 4)
    assert [q.q4nx_kv_page_bytes(*a) for a in ((96, 1, 16), (64, 0, 16), (64, 1, 0), (64, 1, 24), (64, 1, -16), (64, 1025, 16))] == [0] * 6


CACHE_BAD = [(dict(pool=None), 1), (dict(reserved=1), 2), (dict(dim=96), 3), (dict(heads=0), 3), (dict(page=8), 3), (dict(page=24), 3),
             (dict(pages=0), 3), (dict(pages=1 << 31), 3), (dict(nbytes=10 * 64 * 8 * 160 - 1), 4), (dict(pool=P + 8), 5)]
BATCH_BAD = [(dict(a=None), 1), (dict(b=None), 1), (dict(c=None), 1), (dict(batch=0), 3), (dict(batch=1025), 3), (dict(cols=0), 3),
             (dict(tokens=-1), 3), (dict(tokens=1 << 31), 3), (dict(a=P + 2), 5), (dict(c=P + 1), 5)]


def test_cache_entry_points_refuse(q):
    L, by = q.lib, ctypes.byref
    need = L.q4nx_kv_workspace(by(_cache(q)))
    assert need > 16 and L.q4nx_kv_workspace(by(_cache(q, dim=96))) == 0 and L.q4nx_kv_workspace(None) == 0

    def calls(c, b, k=P, v=P, stride=1024, qs=4096, heads=32, window=0, out=P, dt=0, lse=P, ws=P, n=need):
        c, b = None if c is None else by(c), None if b is None else by(b)
        return (L.q4nx_kv_append(c, b, k, v, stride, ws, n, None), L.q4nx_kv_read(c, b, k, v, dt, ws, n, None),
                L.q4nx_kv_attention(c, b, k, qs, heads, 0.1, window, out, dt, lse, ws, n, None))

    assert calls(None, _batch(q)) == (1, 1, 1) and calls(_cache(q), None) == (1, 1, 1)
    for kw, st in CACHE_BAD:
        assert calls(_cache(q, **kw), _batch(q)) == (st,) * 3, kw
    for kw, st in BATCH_BAD:
        assert calls(_cache(q), _batch(q, **kw)) == (st,) * 3, kw
    c, b = _cache(q), _batch(q)
    assert calls(c, b, k=None) == (1, 1, 1) and calls(c, b, v=None)[:2] == (1, 1) and calls(c, b, out=None)[2] == 1
    assert calls(c, b, k=P + 8) == (5, 5, 5) and calls(c, b, v=P + 4)[:2] == (5, 5) and calls(c, b, out=P + 2)[2] == 5
    assert calls(c, b, stride=1016)[0] == 3 and calls(c, b, stride=1028)[0] == 5 and calls(c, b, stride=1 << 41)[0] == 3
    assert calls(c, b, qs=4088)[2] == 3 and calls(c, b, qs=4100)[2] == 5 and calls(c, b, lse=P + 2)[2] == 5
    assert [calls(c, b, heads=h)[2] for h in (0, 12, 1032)] == [3, 3, 3] and calls(c, b, window=-1)[2] == 3
    assert calls(c, b, dt=2)[1:] == (11, 11)
    assert calls(c, b, ws=None) == (7, 7, 7) and calls(c, b, n=need - 1) == (7, 7, 7) and calls(c, b, ws=P + 8) == (5, 5, 5)
    # nothing to do: accepted without a launch
    assert calls(c, _batch(q, tokens=0)) == (0, 0, 0)


def test_cache_entry_points_refuse_is_not_run_beside_a_gpu(monkeypatch):
    import types

    import conftest

    item = types.SimpleNamespace(name="test_cache_entry_points_refuse")
    for gpu in (False, True):
        monkeypatch.setattr(conftest, "gpu_available", lambda: gpu)
        if gpu:
            with pytest.raises(pytest.skip.Exception):
                conftest.pytest_runtest_setup(item)
        else:
            conftest.pytest_runtest_setup(item)
        conftest.pytest_runtest_setup(types.SimpleNamespace(name="test_index_status"))


def test_cache_workspace_holds_what_the_kernels_of_its_size_leave(q):
    # parts of 304 CTAs: 8 rows twice (values, maximum and sum) and 8 per warp; with 64 or
    # 128 channels also the 256 rows of the kernel for many rows, the larger of the two
    for dim in (64, 128, 256):
        few, many = 304 * 8 * (2 * (dim + 2) + 8 * dim) * 4, 304 * 256 * (dim + 2) * 4 if dim < 256 else 0
        head = q.lib.q4nx_kv_workspace(ctypes.byref(_cache(q, dim=dim))) - max(few, many)
        assert 16 + 304 * 4 <= head <= 1 << 16, dim             # error word, counters and records


def test_lora_refuses(q):
    L, by = q.lib, ctypes.byref
    w = q.q4nx_weight(P, 1 << 30, q.Q4NX_Q4_1, 0, 64, 512)
    ws, sc = L.q4nx_gemm_workspace(by(w), 64), L.q4nx_gemm_lora_scratch(by(w), 64)
    assert sc >= 64 * 64 * 4 and L.q4nx_gemm_lora_scratch(by(w), 0) == 0 and L.q4nx_gemm_lora_scratch(by(w), 65) == 0

    def call(w=w, X=P, M=64, a=P, b=P, s=P, na=1 << 30, nb=1 << 30, count=4, rank=16, ids=P, Y=P, dt=0, wsp=P, nws=ws, scp=P, nsc=sc):
        ad = q.q4nx_adapters(a, b, s, na, nb, count, rank)
        return L.q4nx_gemm_lora(by(w), X, M, by(ad), ids, Y, dt, wsp, nws, scp, nsc, None)

    for name in ("X", "a", "b", "s", "ids", "Y"):
        assert call(**{name: None}) == 1, name
    assert L.q4nx_gemm_lora(by(w), P, 64, None, P, P, 0, P, ws, P, sc, None) == 1
    assert call(M=0) == 6 and call(M=65) == 6 and call(count=0) == 3 and call(dt=2) == 11
    assert [call(rank=r) for r in (0, 4, 12, 24, 256)] == [3] * 5
    assert call(na=4 * 16 * 512 * 2 - 1) == 4 and call(nb=4 * 16 * 64 * 2 - 1) == 4
    for name in ("X", "a", "b", "Y", "wsp", "scp"):
        assert call(**{name: P + 8}) == 5, name
    assert call(s=P + 2) == 5 and call(ids=P + 1) == 5
    assert call(wsp=None) == 7 and call(nws=ws - 1) == 7 and call(scp=None) == 7 and call(nsc=sc - 1) == 7
    assert call(w=q.q4nx_weight(P, 1 << 30, q.Q4NX_Q4_1, 0, 63, 512)) == 3
    assert call(w=q.q4nx_weight(P, 1 << 30, q.Q4NX_Q4_K, 0, 64, 512)) == 8        # no tensor-core path for this kind


def test_logprobs_refuses(q):
    def call(x=P, dt=1, M=2, V=100, stride=100, tok=P, top=5, lp=P, ent=P, lse=P, idx=P, tlp=P):
        return q.lib.q4nx_logprobs(x, dt, M, V, stride, tok, top, lp, ent, lse, idx, tlp, None)

    assert call(x=None) == 1 and call(tok=None) == 1 and call(idx=None) == 1 and call(tlp=None) == 1
    assert [call(M=m) for m in (0, 65536)] == [3, 3] and call(V=0, stride=0, top=0) == 3 and call(stride=99) == 3
    assert call(V=1 << 31, stride=1 << 31) == 3
    assert [call(top=t) for t in (-1, 33)] == [3, 3] and call(V=4, top=5) == 3 and call(dt=2) == 11
    for name in ("x", "tok", "lp", "ent", "lse", "idx", "tlp"):
        assert call(**{name: P + 2}) == 5, name
    assert call(x=P + 1, dt=0) == 5


def test_binding_refuses(q):
    cpu = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        q.KVCache(cpu, 128, 1, 16, 1)
    with pytest.raises(ValueError):
        q.KVCache.alloc(1, 1, 96, 16)
    with pytest.raises(ValueError):
        q.Adapters(torch.zeros(1, 8, 256, dtype=torch.bfloat16), torch.zeros(1, 32, 8, dtype=torch.bfloat16), torch.zeros(1))
    with pytest.raises(ValueError):
        q.q4nx_logprobs(torch.zeros(2, 10))


def test_index_status(q):
    assert q.Q4NX_E_INDEX == 12 and q.q4nx_status_str(12) != "unknown status"
