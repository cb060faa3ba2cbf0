"""q4nx_gemm_epilogue against the oracle's product and the epilogue in binary64.

Bound: the sum has the product's own bar (1e-3 A on the CUDA cores, (1e-3 + 2^-9) A on
the tensor cores, A = sum |w x|) and one rounding of the bias's addition; an activation is
within 2^-20 at a number within 2^-21 of the sum, and none is steeper than 1.13; the
product and the addition behind it round once each in binary32; bf16 output: 2^-8."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    import dequant_gemv_gb300

    return dequant_gemv_gb300


def _f64(t):
    return t.double().cpu().numpy()


def few(kind, M):
    return M <= {synth.Q4_1: 2, synth.Q4_K: 4}.get(kind, 1)


_erfc = np.vectorize(math.erfc)


def activated(act, x):
    with np.errstate(over="ignore"):
        return {"none": lambda: x, "relu": lambda: np.maximum(x, 0), "silu": lambda: x / (1 + np.exp(-x)),
                "gelu": lambda: 0.5 * x * _erfc(-x * math.sqrt(0.5)),
                "gelu_tanh": lambda: x / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))}[act]()


class Case:
    def __init__(self, q, kind, N, K, M, seed=0):
        self.N, self.K, self.M, self.kind = N, K, M, kind
        f, self.w = synth.make(kind, N, K, synth.rng(37, seed, N + K))
        self.x = synth.activations(synth.rng(37, 1 + seed, N + K + M), M, K)
        self.W = q.Weight(torch.from_numpy(self.w).to(DEV), kind, N, K)
        self.X = torch.from_numpy(self.x.view(np.int16)).to(DEV).view(torch.bfloat16)
        g = torch.Generator(device=DEV).manual_seed(seed + M)
        n = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
        self.bias, self.mul, self.residual = n(N), n(M, N), n(M, N)
        y, A = oracle.matmul(self.w, kind, N, K, self.x)
        self.y, self.A = y.reshape(M, N), A.reshape(M, N)

    def check(self, out, act="none", bias=None, mul=None, residual=None):
        s = self.y if bias is None else self.y + _f64(bias)
        t = (1e-3 + (0 if few(self.kind, self.M) else 2.0 ** -9)) * self.A
        t = t + 2.0 ** -24 * (np.abs(s) + t)
        v = activated(act, s)
        if act != "none":
            t = 1.13 * (t + 2.0 ** -21 * np.abs(s)) + 2.0 ** -20 * (np.abs(v) + 1.13 * t)
        if mul is not None:
            v = v * _f64(mul)
            t = t * np.abs(_f64(mul)) * (1 + 2.0 ** -24) + 2.0 ** -24 * np.abs(v)
        if residual is not None:
            v = v + _f64(residual)
            t = t + 2.0 ** -24 * (np.abs(v) + t)
        if out.dtype == torch.bfloat16:
            t = t + 2.0 ** -8 * (np.abs(v) + t)
        got = _f64(out)
        assert np.all(np.abs(got - v) <= t), np.max(np.abs(got - v) - t)


ALL = ("bias", "mul", "residual")
SETS = [(), ("bias",), ("mul",), ("residual",), ("bias", "residual"), ("mul", "residual"), ALL]


@pytest.mark.parametrize("M", [1, 2, 3, 8, 33, 64])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_matches(q, act, M):
    c = Case(q, synth.Q4_1, 416, 768, M)
    for names in SETS:
        kw = {n: getattr(c, n) for n in names}
        for dt in ("bf16", "f32"):
            c.check(q.q4nx_gemm_epilogue(c.W, c.X, act=act, out_dtype=dt, **kw), act, **kw)
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("kind,M", [(synth.Q8_KR, 1), (synth.Q8_KR, 17), (synth.Q8_BLK, 64), (synth.Q8_BLK, 1), (synth.Q4_K, 4),
                                    (synth.Q4_K, 2), (synth.Q4_K, 1)])
def test_kinds(q, kind, M):
    c = Case(q, kind, 160, 1280, M)
    kw = {n: getattr(c, n) for n in ALL}
    c.check(q.q4nx_gemm_epilogue(c.W, c.X, act="silu", **kw), "silu", **kw)


# one tile, parts of one, several per CTA (the slot of the operands is used again), a ragged last one
@pytest.mark.parametrize("N,K", [(32, 256), (4096, 256), (32, 12288), (2080, 2560), (24608, 768), (60000, 256)])
@pytest.mark.parametrize("M", [1, 2, 12])
def test_shapes(q, N, K, M):
    c = Case(q, synth.Q4_1, N, K, M)
    for names in (("mul",), ("bias", "residual"), ALL):
        kw = {n: getattr(c, n) for n in names}
        c.check(q.q4nx_gemm_epilogue(c.W, c.X, act="silu", out_dtype="f32", **kw), "silu", **kw)
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("kind,M", [(synth.Q4_1, 1), (synth.Q4_1, 2), (synth.Q4_1, 64), (synth.Q8_KR, 9), (synth.Q4_K, 3)])
def test_nothing_to_do_is_the_product(q, kind, M):
    for N, K in ((416, 768), (20000, 512), (4096, 4096)):
        c = Case(q, kind, N, K, M)
        for dt in ("bf16", "f32"):
            assert torch.equal(q.q4nx_gemm_epilogue(c.W, c.X, out_dtype=dt), q.q4nx_gemm_m64(c.W, c.X, out_dtype=dt))


@pytest.mark.parametrize("M", [1, 2, 20, 64])
def test_parts_of_wider_rows_and_in_place(q, M):
    c = Case(q, synth.Q4_1, 416, 768, M)
    wide = torch.full((M, 3 * 416 + 8), float("nan"), device=DEV, dtype=torch.bfloat16)
    mul, residual = wide[:, 416:832], wide[:, 832:1248]
    mul.copy_(c.mul)
    residual.copy_(c.residual)
    kw = dict(act="gelu", bias=c.bias)
    want = q.q4nx_gemm_epilogue(c.W, c.X, mul=c.mul, residual=c.residual, **kw)
    assert torch.equal(q.q4nx_gemm_epilogue(c.W, c.X, mul=mul, residual=residual, **kw), want)
    for name in ("mul", "residual"):
        side = {n: getattr(c, n).clone() for n in ("mul", "residual")}
        out = q.q4nx_gemm_epilogue(c.W, c.X, out=side[name], **side, **kw)
        assert out is side[name] or out.data_ptr() == side[name].data_ptr()
        assert torch.equal(out, want)
    both = c.mul.clone()                                       # one tensor in all three places
    got = q.q4nx_gemm_epilogue(c.W, c.X, mul=both, residual=both, out=both, **kw)
    assert torch.equal(got, q.q4nx_gemm_epilogue(c.W, c.X, mul=c.mul, residual=c.mul, **kw))


@pytest.mark.parametrize("M", [1, 16])
def test_numbers_at_the_ends(q, M):
    """The sum is the bias (the weight's codes and zeros are zero): tails, signed zeros, infinities, NaN."""
    N, K = 64, 256
    W = q.Weight(torch.zeros(N // 32 * 5120, dtype=torch.uint8, device=DEV), q.Q4NX_Q4_1, N, K)
    X = torch.ones(M, K, device=DEV, dtype=torch.bfloat16)
    some = [0.0, 1e-30, -1e-30, 0.5, -0.5, -3.0, 3.0, -6.0, 6.0, -9.0, -12.0, 30.0, -30.0, -80.0, 1e4, -1e4, 1e15, -1e15, 3e38, -3e38]
    bias = torch.tensor((some * 4)[:N - 3] + [math.inf, -math.inf, math.nan], device=DEV).bfloat16()
    x = _f64(bias)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        got = _f64(q.q4nx_gemm_epilogue(W, X, bias=bias, act=act, out_dtype="f32"))
        with np.errstate(invalid="ignore", over="ignore"):
            steep = 2 * math.sqrt(2 / math.pi) * np.abs(x) * (1 + 3 * 0.044715 * x * x) if act == "gelu_tanh" else x * x + 1 if act == "gelu" else 1
            v = activated(act, x)
            # 2^-21 of the sum moves a tail by up to |x| / act times the slope: the exponent's own derivative
            tol = np.abs(v) * (2.0 ** -20 + 2.0 ** -21 * (1 + np.minimum(steep, 200.0))) + 1e-37
        fin = np.isfinite(x) & (np.abs(x) < 1e10)
        assert np.all(np.abs(got - v)[:, fin] <= tol[fin]), act
        big = np.isfinite(x) & ~fin
        assert np.array_equal(got[:, big], np.broadcast_to(np.maximum(x[big], 0), got[:, big].shape)), act
        assert np.all(got[:, -3] == math.inf) and np.all(np.isnan(got[:, -1])), act
        assert np.all(np.isnan(got[:, -2]) if act != "relu" else got[:, -2] == 0), act


def test_chained_captured_and_on_another_stream(q):
    """A layer's second half as it is called: up, gate with silu and up, down into the residual."""
    H, I, M = 1024, 2048, 24
    up, gate, down = (Case(q, synth.Q4_1, *s, M, seed=i) for i, s in enumerate(((I, H), (I, H), (H, I))))
    x, h0 = up.X, down.residual

    def layer(h):
        u = q.q4nx_gemm_m64(up.W, x)
        g = q.q4nx_gemm_epilogue(gate.W, x, act="silu", mul=u)
        return q.q4nx_gemm_epilogue(down.W, g, residual=h, out=h), u, g

    h, u, g = layer(h0.clone())
    gate.x, gate.X = up.x, x
    y, A = oracle.matmul(gate.w, gate.kind, I, H, up.x)
    gate.y, gate.A = y.reshape(M, I), A.reshape(M, I)
    gate.check(g, "silu", mul=u)
    down.x = g.view(torch.int16).cpu().numpy().view(np.uint16)
    y, A = oracle.matmul(down.w, down.kind, H, I, down.x)
    down.y, down.A = y.reshape(M, H), A.reshape(M, H)
    down.check(h, residual=h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(layer(h0.clone())[0], h)
        into = h0.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer(into)
        for _ in range(3):
            into.copy_(h0)
            graph.replay()
            side.synchronize()
            assert torch.equal(into, h)
    torch.cuda.current_stream().wait_stream(side)
    q.q4nx_check(device=DEV)
