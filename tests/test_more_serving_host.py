"""Host-side checks of the epilogue product (no GPU needed): the documented status for every
bad argument, before any CUDA call."""
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


def test_epilogue_binding_refuses(q):
    w = q.Weight(torch.zeros(5120, dtype=torch.uint8), q.Q4NX_Q4_1, 32, 256)
    with pytest.raises(ValueError, match="activation"):
        q.q4nx_gemm_epilogue(w, torch.zeros(1, 256, dtype=torch.bfloat16), act="swish")
    with pytest.raises(ValueError, match="CUDA"):
        q.q4nx_gemm_epilogue(w, torch.zeros(1, 256, dtype=torch.bfloat16))
