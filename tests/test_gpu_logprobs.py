"""q4nx_logprobs against the formulas in binary64.

Bounds: sum exp(x - m) of positive terms, each off by 2^-21 (exp of a rounded
product) and summed over at most 64 terms in a row and then in a tree: 2^-17 of
itself, so lse is off by 2^-17 and its own rounding, 2^-22 |lse|; a log-probability
by 2^-22 |x| more; the entropy by 2^-16 (1 + sum p |x - m|).  Indexes: equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    import dequant_gemv_gb300

    return dequant_gemv_gb300


def order(x):
    """Indexes by value, largest first, the lower index first among equals (NaN above all)."""
    k = np.where(np.isnan(x), np.inf, x)
    return np.lexsort((np.arange(len(x)), -k, ~np.isnan(x)))


def check(q, t, tokens, top):
    r = q.q4nx_logprobs(t, None if tokens is None else torch.tensor(tokens, dtype=torch.int32, device=DEV), top=top)
    x = t.double().cpu().numpy()
    for m in range(x.shape[0]):
        row = x[m]
        idx = r.top_idx[m].cpu().numpy()
        assert np.array_equal(idx, order(row)[:top])
        lse, ent, tlp = float(r.lse[m]), float(r.entropy[m]), r.top_logprob[m].double().cpu().numpy()
        lp = None if tokens is None else float(r.logprob[m])
        if np.isnan(row).any() or np.isposinf(row).any():
            assert np.isnan(lse) and np.isnan(ent) and np.isnan(tlp).all() and (lp is None or np.isnan(lp))
            continue
        if np.isneginf(row).all():
            assert lse == -np.inf and ent == 0 and np.all(tlp == -np.inf) and (lp is None or lp == -np.inf)
            continue
        mx = row.max()
        e = np.exp(row - mx)
        want = mx + np.log(e.sum())
        p = e / e.sum()
        d = np.where(p > 0, row - mx, 0)
        tol = 2.0 ** -17 + 2.0 ** -22 * abs(want)
        assert abs(lse - want) <= tol
        assert abs(ent - (np.log(e.sum()) - (p * d).sum())) <= 2.0 ** -16 * (1 + (p * -d).sum())
        w = row[idx] - want
        fin = np.isfinite(w)
        assert np.array_equal(tlp[~fin], w[~fin]) and np.all(np.abs(tlp - w)[fin] <= tol + 2.0 ** -22 * np.abs(row[idx][fin]))
        if tokens is not None:
            if not 0 <= tokens[m] < len(row):
                assert np.isnan(lp)
            elif np.isneginf(row[tokens[m]]):
                assert lp == -np.inf
            else:
                assert abs(lp - (row[tokens[m]] - want)) <= tol + 2.0 ** -22 * abs(row[tokens[m]])


def draw(M, V, dtype, seed=0, scale=4.0):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000 + V + M)
    return (torch.randn(M, V, generator=g, device=DEV) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (2, 31), (5, 33), (1, 513), (7, 1000), (1, 32003), (2, 151936), (65, 4099), (40, 20000)])
def test_matches(q, dtype, M, V):
    t = draw(M, V, dtype)
    rng = np.random.default_rng(V)
    for top in (0, 1, 5, 20, 32):
        if top <= V:
            check(q, t, [int(i) for i in rng.integers(0, V, M)], top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [30 * 4, 33 * 8, 65 * 4, 483 * 8, 481 * 16, 514 * 4, 496 * 32])
def test_rows_that_fill_the_last_warps_in_part(q, V, dtype):
    for M in (1, 60, 320):
        t = draw(M, V, dtype, seed=3)
        for top in (17, 32):
            check(q, t, [(7 * m) % V for m in range(M)], top)


@pytest.mark.parametrize("M", [1, 5, 100, 400])
def test_ties_and_masked_entries(q, M):
    g = torch.Generator(device=DEV).manual_seed(M)
    t = torch.randint(-3, 4, (M, 3001), generator=g, device=DEV).float()
    t[:, ::3] = -float("inf")
    check(q, t, [4] * M, 32)
    check(q, t.bfloat16(), [3] * M, 20)


@pytest.mark.parametrize("V", [5, 40, 9000, 151936])
def test_equal_rows_sorted_rows_and_empty_rows(q, V):
    top = min(V, 32)
    t = torch.zeros(5, V, device=DEV)
    t[1] = torch.arange(V, device=DEV) * 2.0 ** -10               # ascending: every element is the best so far
    t[2] = -t[1]
    t[3] = -float("inf")
    t[4] = -float("inf")
    t[4, V // 2] = 3.0
    check(q, t, [0, 1, 2, 3, V // 2], top)
    t = torch.full((1, V), -0.0, device=DEV)
    t[0, ::2] = 0.0                                               # -0 and +0 are equal
    assert np.array_equal(q.q4nx_logprobs(t, top=top).top_idx[0].cpu().numpy(), np.arange(top))


def test_nan_and_infinity(q):
    t = draw(6, 5000, torch.float32)
    t[0, 17] = float("nan")
    t[1, 4999] = float("inf")
    t[2, 3], t[2, 4] = float("inf"), float("nan")
    t[3, :] = float("nan")
    t[4, 7::8] = float("inf")
    check(q, t, [0, 1, 2, 3, 4, 5], 32)


def test_large_and_small_values(q):
    t = draw(4, 4000, torch.float32)
    t[0] *= 1e30
    t[1] *= 1e-30
    t[2] += 3e4
    t[3] -= 1e6
    check(q, t, [1, 2, 3, 4], 10)


def test_rows_at_any_address(q):
    base = draw(9, 3333, torch.float32)
    for lo in (0, 1, 2, 3, 5):
        check(q, base[:, lo:3001 + lo], [7] * 9, 7)
        check(q, base.bfloat16()[:, lo:3001 + lo], [7] * 9, 7)
    check(q, base[::2, 1:4], [0, 1, 2, 3, -1], 3)
    check(q, base[:2], None, 4)


def test_other_stream_and_graph(q):
    t = draw(3, 30000, torch.float32)
    a = q.q4nx_logprobs(t, top=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = q.q4nx_logprobs(t, top=8)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = q.q4nx_logprobs(t, top=8)
    g.replay()
    for x, y, z in zip(a[1:], b[1:], c[1:]):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_binding_refuses(q):
    t = draw(2, 100, torch.float32)
    tok = torch.zeros(2, dtype=torch.int32, device=DEV)
    for args in ((t.half(), tok, 0), (t[0], tok, 0), (t.T, tok, 0), (t, tok.long(), 0), (t, tok[:1], 0), (t, tok, 33), (t, tok, -1)):
        with pytest.raises(ValueError):
            q.q4nx_logprobs(*args)
    with pytest.raises(q.Q4NXError):
        q.q4nx_logprobs(t[:, :3], tok, 5)
