"""Units of one tile's rows, which two tiles take in turn: rows of a warp of which some have no weight left in the
even steps of 64 positions, some in the odd ones, some in neither.

Two channels mark the steps: keys of 100 in the even or the odd ones, queries of 60 in one of them or in none, so that a marked
row's logits of the other steps lie 500 below: e^-500 is 0 in binary32.  Bounds as in tests/test_gpu_kv_shared_accuracy.py:
(2^-15 + 2 * 2^-16 big + 2^-20) A with big the largest sum |q k| scale, where the marks lie; behind a prefix, whose
requests' own tokens go by few rows, 2^-11 + 2^-13 of A more.  A weight below 2^-126 of the row's reference, which lies within 2^8 of
its largest, is 0 in binary32: 9000 of them with values below 16 come to less than 2^-100."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, exact, q  # noqa: F401  (q is a fixture)
from test_gpu_kv_shared import Shared, cross, exact_cross
from test_gpu_kv_shared_accuracy import biggest, within

pytestmark = pytest.mark.gpu


def mark(k, n):
    k[:n, :, :2] = 0
    for p in range(n):
        k[p, :, p // 64 % 2] = 100


class Marked(Case):
    """Queries: row t + head of a request prefers even steps, odd ones, or none, by turns of `turn` rows."""
    turn = 1

    def draw(self, n, heads=None):
        x = super().draw(n, heads)
        if heads is not None:
            kind = (np.arange(n)[:, None] + np.arange(heads)[None]) // self.turn % 3
            x[..., 0], x[..., 1] = 60 * (kind == 0), 60 * (kind == 1)
        return x


class MarkedShared(Shared, Marked):
    pass


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,T", [([64, 65], [70, 66]), ([128, 200], [80, 100]), ([1000, 129], [128, 64]), ([9000], [96])])
@pytest.mark.parametrize("turn", [1, 32])
def test_cross(q, lens, T, dim, turn):  # noqa: F811
    c = Marked(q, lens, lens, 2, dim, 64)
    c.turn = turn
    for b, n in enumerate(lens):
        mark(c.k[b], n)
    c.append_new()
    scale = dim ** -0.5
    qx, out, lse = cross(c, T, 2)
    y, l, A = exact_cross(c, T, qx, scale, 2)
    within(out, lse, y, l, A, biggest(c, qx, scale, 2), np.full(A.shape, 2.0 ** -100))
    again = cross_again(c, T, qx)
    assert torch.equal(again, out)
    q.q4nx_check(device=DEV)


def cross_again(c, T, qx):
    start = torch.tensor(np.concatenate([[0], np.cumsum(T)]), dtype=torch.int32, device=DEV)
    return c.q.q4nx_kv_attention_cross(c.cache, torch.from_numpy(qx).to(DEV).bfloat16(), start, c.tlens, c.table, out_dtype="f32")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shared", [128, 200, 3000])
def test_behind_a_prefix(q, dim, shared):  # noqa: F811
    c = MarkedShared(q, [(shared, [(1 + b % 5, 1) for b in range(50)])], 2, dim, 16, hidden=False)
    for k in c.k:
        mark(k, shared)
    c.fill().append_new()
    qx = c.draw(c.tokens, 4)
    lse = torch.empty(c.tokens, 4, device=DEV)
    out = q.q4nx_kv_attention_shared(c.cache, torch.from_numpy(qx).to(DEV).bfloat16(), c.start, c.tlens, c.table, c.first, c.shared, out_dtype="f32",
                                     lse=lse)
    y, l, A = exact(c, qx, dim ** -0.5, 0, 4)
    within(out, lse, y, l, A, biggest(c, qx, dim ** -0.5, 4), (2.0 ** -11 + 2.0 ** -13) * A + 2.0 ** -100)
    q.q4nx_check(device=DEV)
