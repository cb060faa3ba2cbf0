"""Rows of q4nx_kv_attention_shared whose logits are beyond binary32 on the negative side, in one part or in
both: they weigh nothing there, as in q4nx_kv_attention, whose zeros and -Inf the call has to give where nothing is left.

Queries of -2^116 in every channel, keys of 2^14 (kept exactly): each logit is -2^137 and less times the scale, -Inf in binary32."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, dev, exact, q  # noqa: F401  (q is a fixture)
from test_gpu_kv_shared import Shared, check

pytestmark = pytest.mark.gpu

# the prefixes first, second, and both passes on the tensor cores
FORMS = {"few": [(37, [(2, 1), (20, 1)])], "crowd": [(37, [(2, 1), (20, 1)] * 24)], "prompts": [(37, [(65, 65), (70, 66)])]}


def attend(q, c, qx, heads, name):  # noqa: F811
    lse = torch.full((c.tokens, heads), 7.0, device=DEV)
    groups = (c.first, c.shared) if name == "q4nx_kv_attention_shared" else ()
    return getattr(q, name)(c.cache, dev(qx), c.start, c.tlens, c.table, *groups, out_dtype="f32", lse=lse), lse


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_without_any_weight(q, form, dim):  # noqa: F811
    c = Shared(q, FORMS[form], 2, dim, 16, hidden=False)
    for b in range(len(c.lens)):
        c.k[b][:] = 2.0 ** 14
    c.fill().append_new()
    qx = np.full((c.tokens, 8, dim), -2.0 ** 116, np.float32)
    qx[::2] = c.draw(c.tokens, 8)[::2]                               # and rows like any other
    out, lse = attend(q, c, qx, 8, "q4nx_kv_attention_shared")
    assert torch.all(out[1::2] == 0) and torch.all(lse[1::2] == -torch.inf)
    assert torch.isfinite(out[::2]).all() and torch.isfinite(lse[::2]).all()
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lost", ["shared", "own"])
def test_parts_without_any_weight(q, form, dim, lost):  # noqa: F811
    """Keys of zero in the other part: it alone is left, all its positions alike (the own token's last among them)."""
    c = Shared(q, FORMS[form], 2, dim, 16, hidden=False)
    s = FORMS[form][0][0]
    for b in range(len(c.lens)):
        c.k[b][:] = 0
        if lost == "shared":
            c.k[b][:s] = 2.0 ** 14
        else:
            c.k[b][s:] = 2.0 ** 14
    c.fill().append_new()
    qx = np.full((c.tokens, 8, dim), -2.0 ** 116, np.float32)
    out, lse = attend(q, c, qx, 8, "q4nx_kv_attention_shared")
    check(c, out, lse, *exact(c, qx, dim ** -0.5, 0, 8))
