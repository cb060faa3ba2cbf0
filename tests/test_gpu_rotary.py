"""q4nx_kv_append_rotary: every number is a chain of single binary32 operations, so that
cached values and turned queries are held to equality with the chain on the host; the
table against angles in binary64 (cosine and sine rounded once: 2^-24 each)."""
import math

import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, _bf16, _values, dev, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu


def turn(x, pos, table, interleaved):
    """Rows x [tokens][heads][dim] (binary32) at positions pos, turned in single binary32 steps."""
    half = table.shape[1]
    j = np.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    c, s = table[pos, None, :, 0], table[pos, None, :, 1]
    y = x.astype(np.float32).copy()
    with np.errstate(over="ignore", invalid="ignore"):
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def kept(x):
    """What the cache keeps of turned keys: the rule of the plain append, the range times 1/15 in binary32."""
    v = x.astype(np.float32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        lo, hi = v.min(-1), v.max(-1)
        s = _bf16((hi - lo) * (np.float32(1) / np.float32(15)))
        m = _bf16(lo + np.float32(8) * s)
        c = np.where(s[..., None] == 0, 0, np.clip(np.rint((v - m[..., None]) / s[..., None]), -8, 7))
        bad = (~np.isfinite(v).all(-1) | ~np.isfinite(s) | ~np.isfinite(m))[..., None]
    s, m, c = s.astype(np.float64)[..., None], m.astype(np.float64)[..., None], np.nan_to_num(c).astype(np.float64)
    return np.where(bad, np.nan, c * s + m).reshape(x.shape).astype(np.float32)


def positions(c):
    return np.concatenate([np.arange(n - t, n) for n, t in zip(c.lens, c.new)]) if c.lens else np.zeros(0, int)


def rotary(q, n, dims, interleaved):  # noqa: F811
    r = q.Rotary.make(n, dims, base=1e6, interleaved=interleaved, device=DEV)
    return r, r.table.cpu().numpy()


def run(q, c, heads, dims, interleaved, merged=True, in_place=False):  # noqa: F811
    """The call with the requests' last tokens; (turned queries, expected ones, keys, expected ones, values, expected ones)."""
    pos = positions(c)
    r, table = rotary(q, max(max(c.lens), 1), dims, interleaved)
    qx = c.draw(len(pos), heads)
    ks, vs = (c.stack(x, [n - t for n, t in zip(c.lens, c.new)], c.lens) for x in (c.k, c.v))
    if merged:
        row = dev(np.concatenate([x.reshape(len(pos), -1) for x in (qx, ks, vs)], 1)).unflatten(1, (-1, c.dim))
        qt, kt, vt = row[:, :heads], row[:, heads:heads + c.kv], row[:, heads + c.kv:]
    else:
        qt, kt, vt = dev(qx), dev(ks), dev(vs)
    out = q.q4nx_kv_append_rotary(c.cache, r, qt, kt, vt, c.start, c.tlens, c.table, out=qt if in_place else None)
    assert not in_place or out.data_ptr() == qt.data_ptr()
    k, v = q.q4nx_kv_read(c.cache, len(pos), c.start, c.tlens, c.table, out_dtype="f32")
    return ((out.float().cpu().numpy(), _bf16(turn(qx, pos, table, interleaved))),
            (k.cpu().numpy(), kept(turn(ks, pos, table, interleaved))), (v.cpu().numpy(), _values(vs).astype(np.float32)))


def equal(pairs):
    for got, want in pairs:
        assert got.shape == want.shape and np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("positions,dims,base", [(1, 16, 1e4), (131072, 128, 1e6), (5000, 64, 5e5)])
def test_table(q, positions, dims, base):  # noqa: F811
    t = q.Rotary.make(positions, dims, base=base, device=DEV).table.cpu().numpy().astype(np.float64)
    p, j = np.arange(0, positions, 997, dtype=np.float64)[:, None], np.arange(dims // 2)
    angle = p * base ** (-2.0 * j / dims)
    # pow, and the product's rounding, move a far angle by 4 units in the last place of 64 bits
    tol = 2.0 ** -24 + 2.0 ** -50 * (1 + np.abs(angle))
    assert np.all(np.abs(t[::997, :, 0] - np.cos(angle)) <= tol) and np.all(np.abs(t[::997, :, 1] - np.sin(angle)) <= tol)
    f = torch.linspace(0.001, 3, dims // 2, dtype=torch.float64)
    own = q.Rotary.make(7, dims, frequencies=f, interleaved=True, device=DEV)
    assert own.interleaved and own.table.shape == (7, dims // 2, 2)
    assert abs(float(own.table[6, -1, 1]) - math.sin(18.0)) < 2.0 ** -23


# one token, few, and prompts by blocks; dims whole, in part, and such that partners lie in one group or across two
@pytest.mark.parametrize("dim,dims", [(64, 64), (64, 32), (64, 16), (64, 48), (128, 128), (128, 64), (128, 32), (128, 96), (128, 112),
                                      (256, 256), (256, 192), (256, 64), (256, 16), (256, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kv,heads,lens,new", [(1, 1, [1], [1]), (2, 6, [1, 15, 16, 17, 70, 0, 130], [1, 15, 3, 17, 5, 0, 130]),
                                               (3, 5, [700, 61, 1400, 16, 1000], [700, 60, 1357, 16, 7]), (8, 9, [801, 2000], [801, 190]),
                                               (4, 20, [16 + 7 * b for b in range(64)], [1 + 5 * b % 23 for b in range(64)])])
def test_keeps_the_rule_exactly(q, dim, dims, interleaved, kv, heads, lens, new):  # noqa: F811
    c = Case(q, lens, new, kv, dim, 48, seed=dims)
    equal(run(q, c, heads, dims, interleaved))
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("lens,new", [([40, 33], [1, 2]), ([1500, 900], [1203, 877])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_in_place_and_contiguous(q, lens, new, dim):  # noqa: F811
    for kw in (dict(in_place=True), dict(merged=False), dict(merged=False, in_place=True)):
        equal(run(q, Case(q, lens, new, 4, dim, 16), 12, dim, False, **kw))


@pytest.mark.parametrize("new", [[1, 2], [1000, 600]])
def test_writes_only_its_tokens(q, new):  # noqa: F811
    c = Case(q, [n + 40 for n in new], new, 4, 128, 16, fill=0x5A)
    before = c.cache.pool.clone()
    wide = torch.full((sum(new) + 3, 20, 128), 3.0, device=DEV, dtype=torch.bfloat16)      # three tokens of no request
    out = wide.clone()[:, 2:14]
    r, _ = rotary(q, 2000, 128, False)
    q.q4nx_kv_append_rotary(c.cache, r, wide[:, :12], wide[:, 12:16], wide[:, 16:], c.start, c.tlens, c.table, out=out)
    changed = int((c.cache.pool != before).sum())
    assert 0 < changed <= sum(new) * 4 * 2 * (64 + 16)
    assert torch.all(out[sum(new):] == 3) and torch.all(out._base[:, :2] == 3) and torch.all(out._base[:, 14:] == 3)
    again = c.cache.pool.clone()                                                           # by blocks; without queries by tokens
    assert q.q4nx_kv_append_rotary(c.cache, r, None, wide[:, 12:16], wide[:, 16:], c.start, c.tlens, c.table) is None
    assert torch.equal(c.cache.pool, again)                                                # keys alone: the same bytes
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("n", [400, 1000])
def test_positions_nought_and_without_an_angle_are_the_plain_append(q, n):  # noqa: F811
    c = Case(q, [1, n], [1, n], 16, 128, 64)
    k, v = (dev(c.stack(x, 0, c.lens)) for x in (c.k, c.v))
    q.q4nx_kv_append(c.cache, k, v, c.start, c.tlens, c.table)
    plain = c.cache.pool.clone()
    still = q.Rotary(torch.tensor([1.0, 0.0], device=DEV).repeat(n, 64, 1))
    c.cache.pool.fill_(0xFF)
    qx = torch.randn(n + 1, 3, 128, device=DEV).bfloat16()
    out = q.q4nx_kv_append_rotary(c.cache, still, qx, k, v, c.start, c.tlens, c.table)
    assert torch.equal(out, qx) and torch.equal(c.cache.pool, plain)


@pytest.mark.parametrize("n", [3, 4200])
def test_scale_of_ranges_between_two_steps(q, n):  # noqa: F811
    """Ranges whose 15th part lies midway between two bf16 numbers: turned keys take the product, values the quotient."""
    lo, hi = np.meshgrid(-np.arange(128, 256, dtype=np.float32) / 2 ** 11, np.arange(128, 256, dtype=np.float32) / 64)
    d = hi - lo
    apart = _bf16(d / np.float32(15)) != _bf16(d * (np.float32(1) / np.float32(15)))
    lo, hi = lo[apart], hi[apart]
    assert len(lo) > 20                                       # they are apart for these
    c = Case(q, [n], [n], 4, 128, 16)
    at = np.arange(n * 4 * 4) % len(lo)
    x = np.zeros((n * 4 * 4, 32), np.float32)
    x[:, 5], x[:, 20] = lo[at], hi[at]
    c.k[0] = c.v[0] = x.reshape(n, 4, 128)
    still = q.Rotary(torch.tensor([1.0, 0.0], device=DEV).repeat(n, 64, 1))
    q.q4nx_kv_append_rotary(c.cache, still, None, dev(c.k[0]), dev(c.v[0]), c.start, c.tlens, c.table)
    k, v = (t.cpu().numpy() for t in q.q4nx_kv_read(c.cache, n, c.start, c.tlens, c.table, out_dtype="f32"))
    assert np.array_equal(k, kept(c.k[0])) and np.array_equal(v, _values(c.v[0]).astype(np.float32)) and not np.array_equal(k, v)


# the case whose turned keys showed the two rules apart: one group of 16000
def test_many_tokens_keep_the_rule(q):  # noqa: F811
    c = Case(q, [4001, 3999], [1501, 1999], 8, 128, 64)
    equal(run(q, c, 4, 128, False))


def test_special_numbers(q):  # noqa: F811
    for n in (6, 1600, 2100):
        c = Case(q, [n], [n], 4, 64, 16)
        k = c.k[0]
        k[0, 0, 3] = np.inf                                    # at position 0: inf * 1 - x * 0, and x * 1 + inf * 0 is none
        k[1, 0, 40] = np.nan
        k[2, 0, 0], k[2, 0, 32] = 3.3e38, -3.3e38              # turned beyond binary32
        k[3, 0, :] = 0
        c.k[0] = np.where(np.isfinite(k), _bf16(k), k).astype(np.float32)      # what the call is given
        pairs = run(q, c, 4, 64, False)
        equal(pairs)
        got = pairs[1][0]
        assert np.isnan(got[:2, 0]).all() and np.isnan(got[2, 0, 32:]).all() and not np.isnan(got[2, 0, :32]).any()
        assert not np.isnan(got[3:]).any() and np.all(got[3, 0] == 0)


@pytest.mark.parametrize("new", [5, 900])
def test_tokens_before_the_start(q, new):  # noqa: F811
    """A request with more tokens than its length: what lies before position 0 is neither kept nor written."""
    c = Case(q, [new - 3, new + 20], [new, new], 8, 128, 16)
    r, table = rotary(q, 2000, 128, False)
    x = dev(c.draw(2 * new, 24))
    out = torch.full((2 * new, 8, 128), 9.0, device=DEV, dtype=torch.bfloat16)
    q.q4nx_kv_append_rotary(c.cache, r, x[:, :8], x[:, 8:16], x[:, 16:], c.start, c.tlens, c.table, out=out)
    assert torch.all(out[:3] == 9)
    pos = np.concatenate([np.arange(new - 3), np.arange(20, new + 20)])
    keep = np.r_[3:2 * new]
    host = x.float().cpu().numpy()
    assert np.array_equal(out.float().cpu().numpy()[keep], _bf16(turn(host[keep, :8], pos, table, False)))
    k, _ = q.q4nx_kv_read(c.cache, 2 * new, c.start, c.tlens, c.table, out_dtype="f32")
    assert np.array_equal(k.cpu().numpy()[keep], kept(turn(host[keep, 8:16], pos, table, False)))
    q.q4nx_check(device=DEV)


BAD = [("table", 0, 1, 10 ** 6), ("table", 0, 2, -1), ("lens", 0, None, -3), ("lens", 0, None, 10 ** 6), ("start", 1, None, 10 ** 6),
       ("start", 0, None, -1), ("start", 2, None, 3), ("start", 2, None, 0), ("reach", 0, None, 0)]


@pytest.mark.parametrize("new", [30, 900])
@pytest.mark.parametrize("name,b,i,x", BAD)
def test_reports_what_is_out_of_range(q, new, name, b, i, x):  # noqa: F811
    c = Case(q, [10 + new, 3 + new], [new, new], 8, 64, 16)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    t = {"table": c.table.clone(), "lens": c.tlens.clone(), "start": c.start.clone()}
    if name == "reach":
        r, table = rotary(q, new + 5, 64, False)              # positions of request 0 beyond it
    else:
        r, table = rotary(q, new + 10, 64, False)
        t[name][(b,) if i is None else (b, i)] = x
    kv = dev(c.draw(2 * new, 20))
    before = c.cache.pool.clone()
    out = torch.full((2 * new, 4, 64), 9.0, device=DEV, dtype=torch.bfloat16)
    q.q4nx_kv_append_rotary(c.cache, r, kv[:, 16:], kv[:, :8], kv[:, 8:16], t["start"], t["lens"], t["table"], out=out, ws=ws)
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_check(ws)
    assert e.value.status == q.Q4NX_E_INDEX
    q.q4nx_check(ws)
    if name == "reach":                                       # the tokens that it does not reach stay as they were
        assert torch.all(out[new - 5:new] == 9) and not torch.any((out[:new - 5] == 9).all(-1))
        own = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
        pool = c.cache.pool.clone()
        c.cache.pool.copy_(before)
        was = q.q4nx_kv_read(c.cache, 5, own, c.tlens[:1], c.table[:1], out_dtype="f32")
        c.cache.pool.copy_(pool)
        now = q.q4nx_kv_read(c.cache, 5, own, c.tlens[:1], c.table[:1], out_dtype="f32")
        assert all(torch.equal(x, y) or (torch.isnan(x) == torch.isnan(y)).all() for x, y in zip(was, now))
    out = q.q4nx_kv_append_rotary(c.cache, rotary(q, new + 10, 64, False)[0], kv[:, 16:], kv[:, :8], kv[:, 8:16], c.start, c.tlens, c.table, ws=ws)
    q.q4nx_check(ws)
    assert torch.isfinite(out.float()).all()


def test_captured_and_on_another_stream(q):  # noqa: F811
    c = Case(q, [300, 77], [1, 1], 4, 128, 64)
    r, table = rotary(q, 1000, 128, False)
    x = dev(c.draw(2, 16))
    lens = c.tlens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step = lambda: q.q4nx_kv_append_rotary(c.cache, r, x[:, :8], x[:, 8:12], x[:, 12:], c.start, lens, c.table)  # noqa: E731
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        for n in range(3):
            lens.add_(1)                                      # the graph follows the lengths on the device
            graph.replay()
            side.synchronize()
            pos = np.array([300 + n, 77 + n])
            assert np.array_equal(out.float().cpu().numpy(), _bf16(turn(x[:, :8].float().cpu().numpy(), pos, table, False)))
            k, _ = q.q4nx_kv_read(c.cache, 2, c.start, lens, c.table, out_dtype="f32")
            assert np.array_equal(k.cpu().numpy(), kept(turn(x[:, 8:12].float().cpu().numpy(), pos, table, False)))
    torch.cuda.current_stream().wait_stream(side)
    q.q4nx_check(device=DEV)
