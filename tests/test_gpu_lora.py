"""q4nx_gemm_lora against the oracle's product and the adapters in binary64.

Bound: the product's own bar (1e-3 A on the CUDA cores, (1e-3 + 2^-9) A on the
tensor cores, A = sum |w x|); the adapter's two binary32 sums of exact products,
(cols + rank) 2^-23 of S = |s| |B| (|A| |x|) at most; bf16 output: 2^-8 of the value."""
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


class Case:
    def __init__(self, q, kind, N, K, M, R, count, ids, seed=0):
        self.N, self.K, self.M, self.kind, self.ids = N, K, M, kind, ids
        f, self.w = synth.make(kind, N, K, synth.rng(31, seed, N + K))
        self.x = synth.activations(synth.rng(31, 1 + seed, N + K + M), M, K)
        self.W = q.Weight(torch.from_numpy(self.w).to(DEV), kind, N, K)
        self.X = torch.from_numpy(self.x.view(np.int16)).to(DEV).view(torch.bfloat16)
        g = torch.Generator(device=DEV).manual_seed(seed + R)
        n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.ad = q.Adapters((n(count, R, K) * K ** -0.5).bfloat16(), n(count, N, R).bfloat16(), n(count))
        self.tid = torch.tensor(ids, dtype=torch.int32, device=DEV)

    def exact(self):
        y, A = oracle.matmul(self.w, self.kind, self.N, self.K, self.x)
        y, A = y.reshape(self.M, self.N).copy(), A.reshape(self.M, self.N)
        S = np.zeros_like(y)
        a, b, s, x = _f64(self.ad.a), _f64(self.ad.b), _f64(self.ad.scale), _f64(self.X)
        for m, i in enumerate(self.ids):
            if 0 <= i < len(s):
                y[m] += s[i] * (b[i] @ (a[i] @ x[m]))
                S[m] = abs(s[i]) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[m])))
        return y, A, S

    def check(self, out, few):
        y, A, S = self.exact()
        R = self.ad.a.shape[1]
        tol = (1e-3 + (0 if few else 2.0 ** -9)) * A + (self.K + R) * 2.0 ** -23 * S
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
        got = _f64(out)
        assert np.all(np.abs(got - y) <= tol), np.max(np.abs(got - y) - tol)


def few(kind, M):
    return M <= {synth.Q4_1: 2, synth.Q4_K: 4}.get(kind, 1)


@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("M,block", [(1, False), (2, False), (3, True), (9, False), (33, True), (64, False)])
def test_matches(q, R, M, block):
    count = 5
    ids = [2] * M if block else [(3 * m) % (count + 1) - 1 for m in range(M)]
    c = Case(q, synth.Q4_1, 416, 768, M, R, count, ids)
    for dt in ("bf16", "f32"):
        c.check(q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid, out_dtype=dt), few(c.kind, M))
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("kind,M", [(synth.Q8_KR, 1), (synth.Q8_KR, 17), (synth.Q8_BLK, 64), (synth.Q4_K, 4), (synth.Q4_K, 1)])
def test_kinds(q, kind, M):
    c = Case(q, kind, 160, 1280, M, 16, 64, [(11 * m) % 64 for m in range(M)])
    c.check(q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid), few(kind, M))


@pytest.mark.parametrize("N,K", [(32, 256), (4096, 256), (32, 12288), (2080, 2560)])
def test_shapes(q, N, K):
    M = 12
    c = Case(q, synth.Q4_1, N, K, M, 32, 3, [m % 4 - 1 for m in range(M)])
    c.check(q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid, out_dtype="f32"), False)


@pytest.mark.parametrize("M", [1, 2, 40])
def test_no_adapter_is_the_product(q, M):
    c = Case(q, synth.Q4_1, 256, 512, M, 16, 2, [-1 - m for m in range(M)])
    for dt in ("bf16", "f32"):
        assert torch.equal(q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid, out_dtype=dt), q.q4nx_gemm_m64(c.W, c.X, out_dtype=dt))


def test_many_identical_calls_are_identical(q):
    c = Case(q, synth.Q4_1, 416, 4096, 64, 16, 8, [m % 8 for m in range(64)])
    first = q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid)
    for _ in range(20):
        assert torch.equal(first, q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid))


@pytest.mark.parametrize("M,count,rank", [(64, 64, 16), (33, 1, 64), (9, 4, 8)])
def test_chained_calls_read_what_the_grids_before_wrote(q, M, count, rank):
    # each call's tokens are the last one's output, its ids written just before it: every
    # kernel of a call starts early, and what it reads has to be there all the same
    c = Case(q, synth.Q4_1, 2048, 2048, M, rank, count, [m % (count + 1) - 1 for m in range(M)])

    def steps(wait):
        x, ids, outs = c.X, c.tid, []
        for _ in range(6):
            y = q.q4nx_gemm_lora(c.W, x, c.ad, ids, out_dtype="f32")
            outs.append(y)
            x = (y / y.abs().amax(1, keepdim=True)).bfloat16()
            ids = torch.where(ids + 1 < count, ids + 1, -1)
            if wait:
                torch.cuda.synchronize()
        return outs

    want = steps(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(False)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = steps(False)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
    q.q4nx_check(device=DEV)


def test_adapter_outside_the_pool_adds_nothing_and_is_reported(q):
    c = Case(q, synth.Q4_1, 64, 512, 6, 16, 3, [0, 3, 2, 1 << 30, -1, 1])
    c.check(q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid), False)
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_check(device=DEV)
    assert e.value.status == q.Q4NX_E_INDEX
    q.q4nx_check(device=DEV)


def test_weights_of_different_sizes_share_the_workspace(q):
    cases = [Case(q, synth.Q4_1, N, K, 64, 16, 4, [m % 5 - 1 for m in range(64)]) for N, K in ((4096, 512), (96, 4096), (2048, 2048))]
    for _ in range(2):
        for c in cases:
            c.check(q.q4nx_gemm_lora(c.W, c.X, c.ad, c.tid), False)
    q.q4nx_check(device=DEV)


def test_binding_refuses(q):
    c = Case(q, synth.Q4_1, 64, 512, 4, 16, 3, [0] * 4)
    other = Case(q, synth.Q4_1, 96, 512, 4, 16, 3, [0] * 4)
    for args in ((c.W, c.X, other.ad, c.tid), (c.W, c.X.float(), c.ad, c.tid), (c.W, c.X[:, :256], c.ad, c.tid),
                 (c.W, c.X, c.ad, c.tid.long()), (c.W, c.X, c.ad, c.tid[:3]), (c.W, c.X, c.ad, c.tid.cpu())):
        with pytest.raises(ValueError):
            q.q4nx_gemm_lora(*args)
    with pytest.raises(ValueError):
        q.Adapters(c.ad.a, c.ad.b, c.ad.scale[:2])
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_gemm_lora(c.W, c.X.repeat(17, 1), c.ad, c.tid.repeat(17))
    assert e.value.status == q.Q4NX_E_M
