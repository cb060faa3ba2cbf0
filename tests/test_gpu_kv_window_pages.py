"""Attention over a window where the pages before it have been given back: their table
entries name no page, which is no error, and the results are those of the whole table."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, attend, check, dev, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 48])
@pytest.mark.parametrize("new,group,window", [(1, 2, 40), (1, 2, 17), (3, 4, 1), (5, 3, 100), (40, 2, 33), (150, 1, 23), (70, 4, 65)])
def test_pages_before_the_window_may_be_gone(q, dim, page, new, group, window):  # noqa: F811
    lens = [new, new + 15, new + 16, new + 33, new + 250, new + 1025, new + 1000]
    c = Case(q, lens, [new] * len(lens), 2, dim, page, seed=new + window).fill().append_new()
    heads = 2 * group
    qx, whole, lse, scale = attend(c, heads, window=window)
    check(c, qx, whole, lse, scale, window, heads)
    q.q4nx_check(device=DEV)
    given_back = c.table.clone()
    for b, n in enumerate(lens):
        given_back[b, :max(0, n - new - window + 1) // page] = -1
    qt, lse2 = dev(qx), torch.empty_like(lse)
    out = q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, given_back, scale=scale, window=window, out_dtype="f32", lse=lse2)
    q.q4nx_check(device=DEV)                                # nothing out of range
    assert torch.equal(out, whole) and torch.equal(lse2, lse)
    # one page more is needed, and reported
    b = 5
    first = max(0, lens[b] - new - window + 1) // page
    given_back[b, first] = -1
    q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, given_back, scale=scale, window=window, out_dtype="f32")
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_check(device=DEV)
    assert e.value.status == q.Q4NX_E_INDEX
