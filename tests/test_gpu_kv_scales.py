"""Attention over values whose groups of 32 channels are of very different size.

Bounds, per group: a weight p*scale is rounded by 2^-11 of itself or by 2^-34 of M, the
largest p*scale of the row over tokens and groups, whichever is more, and met by codes of
8 at most: 2^-11 A + 8 n 2^-34 M / sum p for n tokens; the logits' binary32 sums add 2^-13 A
(A = sum p (|(code - 8) scale| + |mid|) / sum p of the channel).  Many rows (pairs of bf16,
no common power of two): 2^-16 A of the pairs and the product left out, 2^-16 A of 132 sums
of 2^-23; a logit is off by 2^-17 of sum |q k| scale for its key's pairs and 2^-19 for its
sums, which moves p and sum p by 2^-16 of it each at most.
"""
import numpy as np
import pytest

from test_gpu_kv import DEV, Case, _bf16, _quantize, _values, attend, exact, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu


def scaled(q, dim, new, steps):  # noqa: F811
    """Values of group g times 2^(-steps * g)."""
    c = Case(q, [700, 90], [new, min(new, 80)], 2, dim, 64, seed=steps)
    f = np.exp2(-float(steps) * (np.arange(dim) // 32)).astype(np.float32)
    c.v = [_bf16(v * f) for v in c.v]
    return c.fill().append_new()


def floors(c, qx, scale, heads):
    """8 n M / sum p of every row in binary64."""
    out, g, at = np.zeros((c.tokens, heads, 1)), heads // c.kv, 0
    for b, (n, t) in enumerate(zip(c.lens, c.new)):
        k, s = _values(c.k[b]), _quantize(c.v[b])[1].max(-1)
        for j in range(t):
            for h in range(heads):
                l = k[:n - t + j + 1, h // g] @ qx[at + j, h].astype(np.float64) * scale
                p = np.exp(l - l.max())
                out[at + j, h] = 8 * len(p) * (p * s[:len(p), h // g]).max() / p.sum()
        at += t
    return out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("steps", [4, 9, 13, 25, 38])
@pytest.mark.parametrize("new", [1, 3])
def test_groups_of_different_scale_few_rows(q, dim, steps, new):  # noqa: F811
    c = scaled(q, dim, new, steps)
    qx, out, lse, scale = attend(c, 4)
    y, l, A = exact(c, qx, scale, 0, 4)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - y) <= (2.0 ** -11 + 2.0 ** -13) * A + 2.0 ** -34 * floors(c, qx, scale, 4))
    assert np.all(np.abs(lse.cpu().numpy() - l) <= 2.0 ** -13 + 2.0 ** -20 * np.abs(l))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("steps", [9, 25, 30])
def test_groups_of_different_scale_many_rows(q, dim, steps):  # noqa: F811
    c = scaled(q, dim, 100, steps)
    qx, out, lse, scale = attend(c, 4, scale=0.2 * dim ** -0.5)
    y, l, A = exact(c, qx, scale, 0, 4)
    big = scale * max(float((np.abs(qx[:, h:h + 1]) @ np.abs(np.concatenate(c.k))[:, h // 2].T).max()) for h in range(4))
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - y) <= (2.0 ** -15 + 2 * 2.0 ** -16 * big) * A)
    assert np.all(np.abs(lse.cpu().numpy() - l) <= 2.0 ** -16 * big + 2.0 ** -17 + 2.0 ** -20 * np.abs(l))
