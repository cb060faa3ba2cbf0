"""Attention of many query rows: calls in which a tile of 128 rows passes steps that the
other one takes, so that the two are at different steps of the same decoded values.

A value kept as NaN shows whether each row read its own step: the rows that see the token
have NaN in its group of 32 channels, all other outputs are finite and within the bounds
of test_gpu_kv (weights 2^-11, logits 2^-13 of A = sum p (|(code - 8) scale| + |mid|) /
sum p; the log-sum 2^-13 + 2^-20 of itself).  Every call is repeated and compared bit for bit.
"""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, _quantize, _values, dev, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu


def formula(c, qx, scale, window, heads):
    """(out with NaN where the row sees one, lse, A) in binary64."""
    outs, As = np.zeros((c.tokens, heads, c.dim)), np.zeros((c.tokens, heads, c.dim))
    lse, g, at = np.full((c.tokens, heads), -np.inf), heads // c.kv, 0
    for b, (n, t) in enumerate(zip(c.lens, c.new)):
        k = _values(c.k[b])
        cv, sv, mv = _quantize(c.v[b])
        odd = np.isnan(sv)                                     # [n][kv][groups]
        sv, mv = np.where(odd, 0, sv), np.where(odd, 0, mv)
        v = (cv * sv[..., None] + mv[..., None]).reshape(c.v[b].shape)
        va = (np.abs(cv * sv[..., None]) + np.abs(mv[..., None])).reshape(c.v[b].shape)
        pos, key = np.arange(n - t, n)[:, None], np.arange(n)[None]
        seen = (key <= pos) & ((key > pos - window) if window else True)
        some = seen.any(1)
        for h in range(heads):
            l = np.where(seen, qx[at:at + t, h].astype(np.float64) @ k[:, h // g].T * scale, -np.inf)
            m = np.where(some, l.max(1, initial=-np.inf), 0)[:, None]
            p = np.exp(l - m)
            z = np.where(some, p.sum(1), 1)
            lse[at:at + t, h] = np.where(some, m[:, 0] + np.log(z), -np.inf)
            nan = (seen.astype(np.float64) @ odd[:, h // g]).repeat(32, 1) > 0
            outs[at:at + t, h] = np.where(nan, np.nan, p @ v[:, h // g] / z[:, None])
            As[at:at + t, h] = p @ va[:, h // g] / z[:, None]
        at += t
    return outs, lse, As


def attend_and_check(c, heads, window=0, times=4):
    c.fill().append_new()
    scale, qx = c.dim ** -0.5, c.draw(c.tokens, heads)
    qt = dev(qx)
    first = None
    for _ in range(times):
        lse = torch.full((c.tokens, heads), 7.0, device=DEV)
        out = c.q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, c.table, scale=scale, window=window, out_dtype="f32", lse=lse)
        c.q.q4nx_check(device=DEV)
        if first is None:
            first = out, lse
        assert torch.equal(out.view(torch.int32), first[0].view(torch.int32)) and torch.equal(lse, first[1])
    y, l, A = formula(c, qx, scale, window, heads)
    got, gl = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(y))
    ok = ~np.isnan(y)
    assert np.all(np.abs(got - y)[ok] <= (2.0 ** -11 + 2.0 ** -13) * A[ok])
    some = np.isfinite(l)
    assert np.array_equal(gl[~some], l[~some]) and np.all(np.abs(gl[some] - l[some]) <= 2.0 ** -13 + 2.0 ** -20 * np.abs(l[some]))
    assert np.all(got[~some] == 0)


def spoil(c, places):
    """A NaN, or an infinity, in the value of (request, position), in a kv head and channel of the generator's choice."""
    for b, p in places:
        c.v[b][p, c.rng.integers(c.kv), c.rng.integers(c.dim)] = c.rng.choice([np.nan, np.inf, -np.inf])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,odd", [(20, [310]), (20, [330]), (1, [300]), (64, [200, 330]), (128, [313, 329]), (200, [140, 141]), (300, [0, 230])])
def test_window_and_one_head_each(q, dim, window, odd):  # noqa: F811
    # the second tile's first visible step is two steps after the first tile's
    c = Case(q, [400], [200], 2, dim, 16, seed=window)
    spoil(c, [(0, p) for p in odd])
    attend_and_check(c, 2, window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [256, 320, 768])
def test_window_of_one_token_from_a_step_s_start(q, dim, length):  # noqa: F811
    # every row sees its own token alone: the tiles have no step in common
    c = Case(q, [length] * 3, [256] * 3, 2, dim, 64, seed=length)
    spoil(c, [(b, length - 256 + p) for b, p in ((0, 0), (0, 128), (1, 127), (1, 255), (2, 64), (2, 191), (2, 192))])
    attend_and_check(c, 2, 1)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,new,requests", [(32, 75, 30), (32, 50, 40), (16, 100, 30)])
def test_units_of_few_rows_before_full_ones(q, dim, heads, new, requests):  # noqa: F811
    # 300 rows per kv head (and 200 of one tile and a part): a CTA takes several whole
    # units, and the second tile has no rows in every other one
    lens = [new + 13 * (b % 9) for b in range(requests)]
    c = Case(q, lens, [new] * requests, 8, dim, 64, seed=new)
    spoil(c, [(b, p) for b in range(requests) for p in (b % 64, lens[b] - 1 - b % 7)])
    attend_and_check(c, heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests,base", [(40, 0), (40, 64), (23, 200)])
def test_causal_units_cut_before_their_last_steps(q, dim, requests, base):  # noqa: F811
    # one query head per kv head: the first tile's rows end two steps before the second
    # tile's, and a CTA may begin with those two steps
    lens = [256 + base + 16 * (b % 5) for b in range(requests)]
    c = Case(q, lens, [256] * requests, 4, dim, 32, seed=base)
    spoil(c, [(b, p) for b in range(requests) for p in ((7 * b) % 64, lens[b] - 100, lens[b] - 256 + (29 * b) % 256)])
    attend_and_check(c, 4)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 100, 150])
def test_requests_of_few_and_of_many_rows(q, dim, window):  # noqa: F811
    # from one row to several units, rows before the first position, nothing in the call
    new = [1, 300, 128, 0, 129, 90, 256, 40, 257, 520, 5, 60] * 3
    lens = [n + (37 * b) % 200 for b, n in enumerate(new)]
    lens[4], lens[9], lens[17] = 100, 390, 60                   # fewer cached than in the call
    c = Case(q, lens, new, 3, dim, 48, seed=window)
    spoil(c, [(b, p) for b, n in enumerate(lens) if n for p in ((11 * b) % n, n - 1 - (5 * b) % min(n, 60))])
    attend_and_check(c, 3, window)
