"""Host-side checks of the epilogue product, the append with a rotation, cross attention and
attention of shared prefixes (no GPU needed): the documented status for every bad argument,
before any CUDA call."""
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


def test_epilogue_refuses(q):
    L, by = q.lib, ctypes.byref
    w = q.q4nx_weight(P, 1 << 30, q.Q4NX_Q4_1, 0, 64, 512)
    ws = L.q4nx_gemm_workspace(by(w), 64)

    def call(w=w, X=P, M=64, bias=P, mul=P, res=P, ms=64, rs=72, act=4, reserved=0, Y=P, dt=0, wsp=P, nws=ws):
        e = q.q4nx_epilogue(bias, mul, res, ms, rs, act, reserved)
        return L.q4nx_gemm_epilogue(None if w is None else by(w), X, M, by(e), Y, dt, wsp, nws, None)

    assert call(w=None) == 1 and call(X=None) == 1 and call(Y=None) == 1
    assert L.q4nx_gemm_epilogue(by(w), P, 64, None, P, 0, P, ws, None) == 1
    assert [call(M=m) for m in (0, 65, -1)] == [6] * 3 and call(reserved=1) == 2
    assert [call(act=a) for a in (-1, 5)] == [8, 8] and call(dt=2) == 11
    assert [call(ms=s) for s in (56, 0, -64, (1 << 38) + 8)] == [3] * 4 and [call(rs=s) for s in (56, 0, -64, (1 << 38) + 8)] == [3] * 4
    assert call(ms=68) == 5 and call(rs=65) == 5
    for name in ("X", "Y", "mul", "res", "wsp"):
        assert call(**{name: P + 8}) == 5, name
    assert call(bias=P + 1) == 5
    assert call(wsp=None) == 7 and call(nws=ws - 1) == 7
    # what is left out is not looked at: it gets as far as the workspace
    assert call(bias=None, mul=None, res=None, ms=0, rs=0, wsp=None) == 7
    assert call(w=q.q4nx_weight(P, 1 << 30, q.Q4NX_Q4_1, 0, 63, 512)) == 3
    assert call(w=q.q4nx_weight(P, 1 << 30, 7, 0, 64, 512)) == 2
    assert call(w=q.q4nx_weight(P, 1 << 30, q.Q4NX_Q4_K, 0, 64, 512)) == 8        # no tensor-core path for this kind


def test_append_rotary_refuses(q):
    L, by = q.lib, ctypes.byref
    cache = dict(pool=P, nbytes=1 << 30, dim=128, heads=8, page=64, reserved=0, pages=10)
    batch = dict(a=P, b=P, c=P, batch=3, cols=4, tokens=3)
    need = L.q4nx_kv_workspace(by(q.q4nx_kv_cache(*cache.values())))

    def call(c=cache, b=batch, table=P, nbytes=1 << 30, positions=1000, dims=128, inter=0, qx=P, qs=4096, heads=32, out=P, os=4096, k=P, v=P,
             kvs=1024, ws=P, n=need):
        r = q.q4nx_rotary(table, nbytes, positions, dims, inter)
        return L.q4nx_kv_append_rotary(None if c is None else by(q.q4nx_kv_cache(*c.values())), None if b is None else by(q.q4nx_kv_batch(*b.values())),
                                       by(r), qx, qs, heads, out, os, k, v, kvs, ws, n, None)

    assert call(c=None) == 1 and call(b=None) == 1 and call(c=dict(cache, dim=96)) == 3 and call(b=dict(batch, batch=0)) == 3
    assert call(b=dict(batch, b=None)) == 1 and call(c=dict(cache, nbytes=10)) == 4 and call(c=dict(cache, reserved=3)) == 2
    assert L.q4nx_kv_append_rotary(by(q.q4nx_kv_cache(*cache.values())), by(q.q4nx_kv_batch(*batch.values())), None, P, 4096, 32, P, 4096, P, P,
                                   1024, P, need, None) == 1
    for name in ("table", "k", "v", "out"):
        assert call(**{name: None}) == 1, name
    assert [call(inter=i) for i in (-1, 2)] == [8, 8]
    assert [call(dims=d) for d in (0, 8, 24, 144, -16)] == [3] * 5 and [call(positions=p) for p in (0, -1, 1 << 31)] == [3] * 3
    assert call(nbytes=1000 * 512 - 1) == 4 and call(dims=16, nbytes=1000 * 64 - 1) == 4
    assert [call(heads=h) for h in (0, -1, 1025)] == [3] * 3
    assert call(kvs=1016) == 3 and call(kvs=1028) == 5 and call(kvs=1 << 41) == 3
    assert call(qs=4088) == 3 and call(qs=4100) == 5 and call(os=4088) == 3 and call(os=4100) == 5 and call(os=1 << 41) == 3
    for name in ("table", "qx", "out", "k", "v", "ws"):
        assert call(**{name: P + 8}) == 5, name
    assert call(ws=None) == 7 and call(n=need - 1) == 7
    # without queries theirs are not looked at; nothing to do is accepted without a launch
    assert call(qx=None, out=None, heads=0, qs=0, os=3, ws=None) == 7 and call(b=dict(batch, tokens=0)) == 0
    assert call(heads=5, qs=640, os=640, b=dict(batch, tokens=0)) == 0            # any number of heads


def test_attention_cross_and_shared_refuse(q):
    L, by = q.lib, ctypes.byref
    cache = dict(pool=P, nbytes=1 << 30, dim=128, heads=8, page=64, reserved=0, pages=10)
    batch = dict(a=P, b=P, c=P, batch=3, cols=4, tokens=3)
    c0 = q.q4nx_kv_cache(*cache.values())
    need, sc = L.q4nx_kv_workspace(by(c0)), L.q4nx_kv_attention_shared_scratch(by(c0), 3, 32)
    assert sc >= 3 * 32 * (128 * 4 + 8)
    assert [L.q4nx_kv_attention_shared_scratch(*a) for a in ((None, 3, 32), (by(c0), -1, 32), (by(c0), 1 << 31, 32), (by(c0), 3, 0), (by(c0), 3, 1025),
                                                             (by(q.q4nx_kv_cache(*dict(cache, dim=96).values())), 3, 32))] == [0] * 6
    assert L.q4nx_kv_attention_shared_scratch(by(c0), 100000, 32) - sc >= 99000 * 32 * 520

    def calls(c=cache, b=batch, qx=P, qs=4096, heads=32, out=P, dt=0, lse=P, ws=P, n=need, first=P, shared=P, count=2, reserved=0, scp=P, nsc=sc):
        c, b = None if c is None else by(q.q4nx_kv_cache(*c.values())), None if b is None else by(q.q4nx_kv_batch(*b.values()))
        g = q.q4nx_kv_groups(first, shared, count, reserved)
        return (L.q4nx_kv_attention_shared(c, b, by(g), qx, qs, heads, 0.1, out, dt, lse, ws, n, scp, nsc, None),)

    def both(**kw):
        c, b = kw.pop("c", cache), kw.pop("b", batch)
        a = dict(qx=P, qs=4096, heads=32, out=P, dt=0, lse=P, ws=P, n=need)
        a.update(kw)
        cross = L.q4nx_kv_attention_cross(None if c is None else by(q.q4nx_kv_cache(*c.values())), None if b is None else by(q.q4nx_kv_batch(*b.values())),
                                          a["qx"], a["qs"], a["heads"], 0.1, a["out"], a["dt"], a["lse"], a["ws"], a["n"], None)
        return cross, *calls(c=c, b=b, **kw)

    assert both(c=None) == (1, 1) and both(b=None) == (1, 1) and both(qx=None) == (1, 1) and both(out=None) == (1, 1)
    assert both(c=dict(cache, dim=96)) == (3, 3) and both(b=dict(batch, batch=1025)) == (3, 3) and both(b=dict(batch, c=P + 2)) == (5, 5)
    assert [both(heads=h) for h in (0, 12, 1032)] == [(3, 3)] * 3 and both(qs=4088) == (3, 3) and both(qs=4100) == (5, 5)
    assert both(dt=2) == (11, 11) and both(lse=P + 2) == (5, 5) and both(qx=P + 8) == (5, 5) and both(out=P + 2) == (5, 5)
    assert both(ws=None) == (7, 7) and both(n=need - 1) == (7, 7) and both(ws=P + 8) == (5, 5)
    assert calls(first=None) == (1,) and calls(shared=None) == (1,) and calls(reserved=1) == (2,)
    assert [calls(count=n) for n in (0, -1, 1025)] == [(3,)] * 3 and calls(first=P + 2) == (5,) and calls(shared=P + 1) == (5,)
    assert calls(scp=None) == (7,) and calls(nsc=sc - 1) == (7,) and calls(scp=P + 8) == (5,)
    assert L.q4nx_kv_attention_shared(by(c0), by(q.q4nx_kv_batch(*batch.values())), None, P, 4096, 32, 0.1, P, 0, P, P, need, P, sc, None) == 1
    # nothing to do: accepted without a launch
    assert both(b=dict(batch, tokens=0)) == (0, 0)


def test_rotary_binding_refuses(q):
    for t in (torch.zeros(4, 8, 2), torch.zeros(4, 8, 2, dtype=torch.float64), torch.zeros(4, 16)):
        with pytest.raises(ValueError):
            q.Rotary(t)
    with pytest.raises(ValueError, match="frequencies"):
        q.Rotary.make(4, 32, frequencies=torch.ones(15, dtype=torch.float64), device="cpu")


def test_epilogue_binding_refuses(q):
    w = q.Weight(torch.zeros(5120, dtype=torch.uint8), q.Q4NX_Q4_1, 32, 256)
    with pytest.raises(ValueError, match="activation"):
        q.q4nx_gemm_epilogue(w, torch.zeros(1, 256, dtype=torch.bfloat16), act="swish")
    with pytest.raises(ValueError, match="CUDA"):
        q.q4nx_gemm_epilogue(w, torch.zeros(1, 256, dtype=torch.bfloat16))
