"""q4nx_kv_attention_shared and q4nx_kv_attention_cross against the formulas in binary64.

Bounds as for q4nx_kv_attention (tests/test_gpu_kv.py): an output is off by at most
2^-11 + 2^-13 of A = sum p (|(code-8) scale| + |mid|) / sum p, the larger of the two kernels' bounds;
joining the two parts of a row costs a few roundings of binary32 and two powers of two of 2^-22:
2^-20 of A.  bf16 output: 2^-8 of the value.  lse: 2^-13 + 2^-20 |lse|."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, _quantize, attend, dev, exact, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Shared(Case):
    """Groups of requests: [(shared tokens, [(tokens behind them, those of the call among them), ..]), ..].

    A group's first request has the prefix in its pages; the others' tables name its whole pages, or nothing
    (hidden), and their copy of the page where it ends holds NaN in the prefix's place."""

    def __init__(self, q, groups, kv, dim, page, seed=0, hidden=True):  # noqa: F811
        lens = [s + own for s, reqs in groups for own, _ in reqs]
        new = [t for _, reqs in groups for _, t in reqs]
        super().__init__(q, lens, new, kv, dim, page, seed=seed)
        self.first = ints(np.concatenate([[0], np.cumsum([len(r) for _, r in groups])]))
        self.shared = ints([s for s, _ in groups])
        table, self.skip, b = self.table.cpu().numpy(), [], 0
        for s, reqs in groups:
            for i in range(len(reqs)):
                if i > 0:
                    self.k[b][:s], self.v[b][:s] = self.k[b - i][:s], self.v[b - i][:s]
                    table[b, :s // page] = -1 if hidden else table[b - i, :s // page]
                self.skip.append(s if i > 0 else 0)
                b += 1
        self.table = torch.from_numpy(table).to(DEV)

    def fill(self):
        old = [max(s, n - t) for n, t, s in zip(self.lens, self.new, self.skip)]
        self.append(self.stack(self.k, self.skip, old), self.stack(self.v, self.skip, old), [o - s for o, s in zip(old, self.skip)], old)
        return self


def run(c, heads, out_dtype="f32", ws=None, first=None, shared=None, qx=None, out=None):
    qx = c.draw(c.tokens, heads) if qx is None else qx
    row = np.concatenate([qx.reshape(c.tokens, -1), c.draw(c.tokens, 2 * c.kv).reshape(c.tokens, -1)], 1)
    qt = dev(row)[:, :heads * c.dim].unflatten(1, (heads, c.dim))
    lse = torch.full((c.tokens, heads), 7.0, device=DEV)
    out = c.q.q4nx_kv_attention_shared(c.cache, qt, c.start, c.tlens, c.table, c.first if first is None else first,
                                       c.shared if shared is None else shared, out_dtype=out_dtype, lse=lse, ws=ws, out=out)
    return qx, out, lse


def check(c, out, lse, y, l, A):
    got, gl = out[:len(y)].float().cpu().numpy().astype(np.float64), lse[:len(y)].cpu().numpy().astype(np.float64)
    tol = (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -20) * A
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
    empty = np.isinf(l)
    assert np.array_equal(np.isneginf(gl), empty) and not np.isnan(got).any()
    assert np.all(got[empty] == 0)
    assert np.all(np.abs(got - y) <= tol), np.max(np.abs(got - y) - tol)
    assert np.all(np.abs(gl - l)[~empty] <= 2.0 ** -13 + 2.0 ** -20 * np.abs(l[~empty]))


GROUPS = {
    # one token each, prefixes that end inside a block, at a block, at a page, in the first block
    "decode": [(37, [(1, 1), (5, 1), (40, 1)]), (64, [(3, 1), (17, 1)]), (96, [(1, 1)]), (3, [(2, 1), (90, 1), (16, 1)])],
    # groups that share nothing, of one request, without a token in the call, with tokens before the first position
    "odd": [(0, [(5, 1), (3, 7), (1, 1)]), (50, [(9, 2)]), (48, [(4, 0), (7, 3)]), (33, [(0, 0), (2, 0)]), (0, [(0, 0)]), (16, [(6, 6), (5, 5)])],
    # many rows a group and few a request; and long enough to be cut between CTAs
    "crowd": [(700, [(1 + 13 * i, 1) for i in range(33)]), (1999, [(2 + i, 2) for i in range(17)])],
    "long": [(9001, [(300, 1), (20, 1), (1, 1), (77, 1)])],
    # prompts behind a prefix: many rows a request too
    "prompts": [(333, [(65, 65), (200, 97)]), (80, [(70, 64)])],
}


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,group,page", [(1, 1, 16), (2, 4, 64), (2, 3, 48), (1, 8, 32)])
@pytest.mark.parametrize("name", list(GROUPS))
def test_shared_matches(q, name, kv, group, page, dim):  # noqa: F811
    c = Shared(q, GROUPS[name], kv, dim, page, seed=group).fill().append_new()
    want = None
    for dt in ("f32", "bf16"):
        qx, out, lse = run(c, kv * group, dt, qx=want and want[0])
        want = want or (qx, exact(c, qx, dim ** -0.5, 0, kv * group))
        check(c, out, lse, *want[1])
    again = run(c, kv * group, "bf16", qx=qx)
    assert torch.equal(again[1], out) and torch.equal(again[2], lse)
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_shared_many_rows_and_units(q, dim):  # noqa: F811
    # more than 256 rows a group, several units and kv heads, a prefix cut between CTAs
    c = Shared(q, [(2500, [(1 + 29 * i, 1 + i % 3) for i in range(40)]), (1, [(30, 1)])], 4, dim, 256, hidden=False).fill().append_new()
    qx, out, lse = run(c, 32)
    check(c, out, lse, *exact(c, qx, dim ** -0.5, 0, 32))


def test_shared_without_prefixes_is_the_attention(q):  # noqa: F811
    c = Shared(q, [(0, [(n, 1) for n in (1, 40, 700)]), (0, [(33, 1)])], 2, 128, 64).fill().append_new()
    qx, want, lse, scale = attend(c, 8)
    _, out, l = run(c, 8, qx=qx)
    assert torch.equal(out, want) and torch.equal(l, lse)


def test_shared_out_lse_and_rows_of_no_request(q):  # noqa: F811
    c = Shared(q, GROUPS["decode"], 2, 128, 16).fill().append_new()
    c.tokens += 3
    qx = c.draw(c.tokens, 4)
    given = torch.full((c.tokens, 4, 128), 5.0, device=DEV, dtype=torch.bfloat16)
    _, out, lse = run(c, 4, "bf16", qx=qx, out=given)
    assert out.data_ptr() == given.data_ptr()
    assert torch.all(out[-3:] == 5) and torch.all(lse[-3:] == 7) and not torch.any((out[:-3] == 5).all(-1))
    qt = dev(qx)
    assert torch.equal(q.q4nx_kv_attention_shared(c.cache, qt, c.start, c.tlens, c.table, c.first, c.shared)[:-3], out[:-3])


@pytest.mark.parametrize("dim", [128, 256])
def test_shared_nan_stays_in_its_group(q, dim):  # noqa: F811
    for name in ("decode", "crowd"):
        c = Shared(q, GROUPS[name], 2, dim, 16)
        c.k[0][5, 1, 3] = np.nan
        c.v[0][9, 0, 40] = np.nan
        c.fill().append_new()
        _, out, _ = run(c, 4)
        bad = torch.isnan(out.view(c.tokens, 2, 2, dim))
        rows = int(c.start[int(c.first[1])])
        assert bad[:rows, 1].all() and bad[:rows, 0, :, 32:64].all() and not bad[:rows, 0, :, :32].any() and not bad[:rows, 0, :, 64:].any()
        assert not bad[rows:].any()


BAD = [("shared", 0, -1), ("shared", 0, 10 ** 6), ("shared", 0, 39), ("first", 0, 1), ("first", 1, 5), ("first", 1, -3), ("first", 2, 3),
       ("first", 2, 10 ** 6), ("table", (0, 1), 10 ** 6), ("table", (0, 0), -1), ("lens", 3, -1), ("lens", 2, 10 ** 6), ("start", 2, 10 ** 6), ("start", 0, -4)]


@pytest.mark.parametrize("name,at,x", BAD)
@pytest.mark.parametrize("count,dim", [(1, 64), (24, 64), (24, 256)])
def test_shared_reports_what_is_out_of_range(q, name, at, x, count, dim):  # noqa: F811
    """Two groups of two requests (24: of many rows): reported, and nothing else is disturbed."""
    c = Shared(q, [(37, [(2, 1), (20, 1)] * count), (50, [(1, 1), (4, 1)])], 2, dim, 16).fill().append_new()
    qx, good, _ = run(c, 8)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    t = dict(shared=c.shared.clone(), first=c.first.clone(), table=c.table, lens=c.tlens, start=c.start)
    keep = c.table, c.tlens, c.start
    c.table, c.tlens, c.start = c.table.clone(), c.tlens.clone(), c.start.clone()
    if name in ("table", "lens", "start"):
        dict(table=c.table, lens=c.tlens, start=c.start)[name][at] = x
    else:
        t[name][at] = x
    run(c, 8, ws=ws, qx=qx, first=t["first"], shared=t["shared"])
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_check(ws)
    assert e.value.status == q.Q4NX_E_INDEX
    c.table, c.tlens, c.start = keep
    _, out, _ = run(c, 8, ws=ws, qx=qx)
    assert torch.equal(out, good)
    q.q4nx_check(ws)


@pytest.mark.parametrize("name,dim", [("decode", 128), ("crowd", 128), ("prompts", 128), ("crowd", 256), ("prompts", 256)])
def test_shared_captured_on_other_streams_and_workspaces(q, name, dim):  # noqa: F811
    """Two captured graphs of two streams, replayed at once: their workspaces and scratch are their own."""
    cases = [Shared(q, GROUPS[name], 2, dim, 16, seed=s).fill().append_new() for s in (1, 2)]
    qs = [c.draw(c.tokens, 8) for c in cases]
    want = [run(c, 8, qx=x)[1].clone() for c, x in zip(cases, qs)]
    graphs, outs = [], []
    for c, x in zip(cases, qs):
        qt, s = dev(x), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call = lambda: q.q4nx_kv_attention_shared(c.cache, qt, c.start, c.tlens, c.table, c.first, c.shared, out_dtype="f32")  # noqa: E731,B023
        with torch.cuda.stream(s):
            assert torch.equal(call(), want[len(graphs)])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(call())
            graphs.append((g, s, qt))
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # calls of different shapes one after the other on one stream and one workspace
    for _ in range(3):
        for c, x, w in zip(cases, qs, want):
            assert torch.equal(run(c, 8, qx=x)[1], w)
            other = Shared(q, GROUPS["long"], 1, 256, 32).fill().append_new()
            run(other, 2)
    q.q4nx_check(device=DEV)


# ---------------------------------------------------------------------- cross --

def exact_cross(c, T, qx, scale, heads):
    y, l, A = np.zeros((len(qx), heads, c.dim)), np.full((len(qx), heads), -np.inf), np.zeros((len(qx), heads, c.dim))
    g, at = heads // c.kv, 0
    for b, t in enumerate(T):
        if c.lens[b] > 0 and t > 0:
            ck, sk, mk = _quantize(c.k[b])
            cv, sv, mv = _quantize(c.v[b])
            k = (ck * sk[..., None] + mk[..., None]).reshape(c.k[b].shape)
            v = (cv * sv[..., None] + mv[..., None]).reshape(c.v[b].shape)
            va = (np.abs(cv * sv[..., None]) + np.abs(mv[..., None])).reshape(c.v[b].shape)
            for h in range(heads):
                x = qx[at:at + t, h].astype(np.float64) @ k[:, h // g].T * scale
                m = x.max(1, keepdims=True)
                p = np.exp(x - m)
                z = p.sum(1, keepdims=True)
                l[at:at + t, h] = (m + np.log(z))[:, 0]
                y[at:at + t, h], A[at:at + t, h] = p / z @ v[:, h // g], p / z @ va[:, h // g]
        at += t
    return y, l, A


def cross(c, T, heads, out_dtype="f32", extra=0, **kw):
    qx = c.draw(sum(T) + extra, heads)
    lse = torch.full((len(qx), heads), 7.0, device=DEV)
    out = c.q.q4nx_kv_attention_cross(c.cache, dev(qx), ints(np.concatenate([[0], np.cumsum(T)])), c.tlens, c.table, out_dtype=out_dtype, lse=lse, **kw)
    return qx, out, lse


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,group,page", [(1, 1, 16), (8, 1, 64), (2, 4, 48), (1, 16, 32)])
@pytest.mark.parametrize("T", [[1] * 8, [3, 0, 1, 2, 5, 1, 0, 9], [70, 1, 90, 0, 65, 129, 64, 300]])
def test_cross_matches(q, T, kv, group, page, dim):  # noqa: F811
    lens = [1, 16, 0, 70, 250, 33, 15, 1025]
    c = Case(q, lens, lens, kv, dim, page, seed=group).append_new()
    for dt in ("f32", "bf16"):
        qx, out, lse = cross(c, T, kv * group, dt)
        check(c, out, lse, *exact_cross(c, T, qx, dim ** -0.5, kv * group))
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("dim", [128, 256])
def test_cross_long_and_rows_of_no_request(q, dim):  # noqa: F811
    c = Case(q, [20000, 3], [20000, 3], 1, dim, 256).append_new()
    for T in ([1, 1], [80, 70]):
        qx, out, lse = cross(c, T, 4, extra=2)
        check(c, out, lse, *exact_cross(c, T, qx[:-2], dim ** -0.5, 4))
        assert torch.all(lse[-2:] == 7)


@pytest.mark.parametrize("dim", [128, 256])
def test_cross_nan_and_what_lies_behind_the_length(q, dim):  # noqa: F811
    # the block in which a cache ends holds NaN behind it (the pool's fill); a NaN key of one request stays there
    for T in ([1, 2], [66, 100]):
        c = Case(q, [5, 40], [5, 40], 2, dim, 16)
        c.k[1][39, 0, 0] = np.nan
        c.append_new()
        _, out, _ = cross(c, T, 2)
        assert torch.isfinite(out[:T[0]]).all() and torch.isnan(out[T[0]:, 0]).all() and torch.isfinite(out[T[0]:, 1]).all()


@pytest.mark.parametrize("T,dim", [([1, 1], 64), ([90, 70], 64), ([90, 70], 256)])
@pytest.mark.parametrize("name,at,x", [("table", (0, 1), 10 ** 6), ("table", (1, 0), -1), ("lens", 0, -3), ("lens", 1, 10 ** 6), ("start", 1, 10 ** 6),
                                       ("start", 2, 0)])
def test_cross_reports_what_is_out_of_range(q, T, dim, name, at, x):  # noqa: F811
    c = Case(q, [40, 33], [40, 33], 2, dim, 16).append_new()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    t = dict(start=ints(np.concatenate([[0], np.cumsum(T)])), lens=c.tlens.clone(), table=c.table.clone())
    qt = dev(c.draw(sum(T), 4))
    call = lambda: q.q4nx_kv_attention_cross(c.cache, qt, t["start"], t["lens"], t["table"], ws=ws)  # noqa: E731
    good, was = call(), t[name][at].clone()
    q.q4nx_check(ws)
    t[name][at] = x
    call()
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_check(ws)
    assert e.value.status == q.Q4NX_E_INDEX
    t[name][at] = was
    assert torch.equal(call(), good)
    q.q4nx_check(ws)
