"""Cross attention and shared prefixes of many rows: the accuracy of the bf16 pairs, at 64, 128 and 256 channels,
in units of one tile's rows (taken by two tiles in turn, or the one tile of 256 channels) and of more.

Bounds as in tests/test_gpu_kv_scales.py for many rows: (2^-15 + 2 * 2^-16 big) A, big = the largest sum |q k| scale
(at 256 channels a logit's 32 sums of 2^-23 are 2^-18 of it, with 2^-17 of the keys' pairs still below 2^-16); up to 704
positions, 132 sums.  Joining two parts: 2^-20 A.

Where a request's own part goes by few rows (fp16 weights), that part adds what is its own: with A_o and s_o the
part of A and of the weights that its positions have, 2^-11 A_o of the weights' rounding and 8 n 2^-34 M / sum p (n positions, M the
largest p * value scale among them), and 2^-14 (A_o + s_o A) of its logits' sums."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, _bf16, _quantize, exact, q  # noqa: F401  (q is a fixture)
from test_gpu_kv_shared import Shared, cross, exact_cross, run

pytestmark = pytest.mark.gpu


def scaled(c, steps):
    """Values of group g times 2^(-steps * g)."""
    f = np.exp2(-float(steps) * (np.arange(c.dim) // 32)).astype(np.float32)
    c.v = [_bf16(v * f) for v in c.v]
    return c


def biggest(c, qx, scale, heads):
    g = heads // c.kv
    return scale * max(float((np.abs(qx[:, h]) @ np.abs(np.concatenate(c.k))[:, h // g].T).max()) for h in range(heads))


def within(out, lse, y, l, A, big, more=0.0):
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - y) <= (2.0 ** -15 + 2 * 2.0 ** -16 * big + 2.0 ** -20) * A + more)
    assert np.all(np.abs(lse.cpu().numpy() - l) <= 2.0 ** -16 * big + 2.0 ** -17 + 2.0 ** -20 * np.abs(l) + (2.0 ** -13 if np.ndim(more) else 0))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("steps", [0, 9, 25])
@pytest.mark.parametrize("T", [[100, 70], [40, 33], [64, 1]])
def test_cross(q, dim, steps, T):  # noqa: F811
    c = scaled(Case(q, [700, 90], [700, 90], 2, dim, 64, seed=steps), steps).append_new()
    scale = 0.2 * dim ** -0.5
    qx, out, lse = cross(c, T, 8, scale=scale)
    within(out, lse, *exact_cross(c, T, qx, scale, 8), biggest(c, qx, scale, 8))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("steps", [0, 9, 25])
def test_prompts_behind_prefixes(q, dim, steps):  # noqa: F811
    c = scaled(Shared(q, [(600, [(100, 100), (60, 60)]), (333, [(70, 66)])], 2, dim, 48, seed=steps), steps).fill().append_new()
    c_scale = 0.2 * dim ** -0.5
    qx = c.draw(c.tokens, 4)
    lse = torch.empty(c.tokens, 4, device=DEV)
    out = q.q4nx_kv_attention_shared(c.cache, torch.from_numpy(qx).to(DEV).bfloat16(), c.start, c.tlens, c.table, c.first, c.shared, scale=c_scale,
                                     out_dtype="f32", lse=lse)
    within(out, lse, *exact(c, qx, c_scale, 0, 4), biggest(c, qx, c_scale, 4))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("count", [33, 100])
def test_answers_behind_a_prefix(q, dim, count):  # noqa: F811
    """One token of every request: the prefix by pairs (66 rows a kv head, and 200), the own tokens by few rows."""
    s, heads = 650, 4
    c = Shared(q, [(s, [(1 + b % 40, 1) for b in range(count)])], 2, dim, 48, seed=count).fill().append_new()
    qx, out, lse = run(c, heads)
    scale = dim ** -0.5
    y, l, A = exact(c, qx, scale, 0, heads)
    more = np.zeros((count, heads, dim))
    for b in range(count):
        ck, sk, mk = _quantize(c.k[b][s:])
        cv, sv, mv = _quantize(c.v[b][s:])
        k = (ck * sk[..., None] + mk[..., None]).reshape(c.k[b][s:].shape)
        va = (np.abs(cv * sv[..., None]) + np.abs(mv[..., None])).reshape(k.shape)
        for h in range(heads):
            p = np.exp(k[:, h // 2] @ qx[b, h].astype(np.float64) * scale - l[b, h])       # its share of all weights
            A_o = p @ va[:, h // 2]
            M = (p[:, None] * sv[:, h // 2]).max()
            more[b, h] = 2.0 ** -11 * A_o + 8 * len(p) * 2.0 ** -34 * M + 2.0 ** -14 * (A_o + p.sum() * A[b, h])
    within(out, lse, y, l, A, biggest(c, qx, scale, heads), more)
