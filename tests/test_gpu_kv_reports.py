"""Each cache call reports an index out of range by itself: the workspace is clear before
every one of them."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, attend, dev, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu

# (array, request, column or None, value, calls that meet it)
ALL = ("append", "read", "attention")
BAD = [("table", 0, 1, 10 ** 6, ("attention",)), ("table", 0, 2, -1, ALL), ("lens", 0, None, -3, ALL), ("lens", 0, None, 10 ** 6, ALL),
       ("start", 1, None, 10 ** 6, ALL), ("start", 0, None, -1, ALL), ("start", 2, None, 3, ALL), ("start", 2, None, 0, ALL)]


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("name,b,i,x,calls", BAD)
def test_every_call_reports(q, new, name, b, i, x, calls):  # noqa: F811
    c = Case(q, [39 + new, 29 + new], [new, new], 2, 64, 16).fill().append_new()
    qx, good, _, scale = attend(c, 4)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    t = {"table": c.table.clone(), "lens": c.tlens.clone(), "start": c.start.clone()}
    if i is None:
        t[name][b] = x
    else:
        t[name][b, i] = x
    k, v = dev(c.draw(2 * new)), dev(c.draw(2 * new))
    args = t["start"], t["lens"], t["table"]
    for call in ALL:
        if call == "append":
            q.q4nx_kv_append(c.cache, k, v, *args, ws=ws)
        elif call == "read":
            q.q4nx_kv_read(c.cache, c.tokens, *args, ws=ws)
        else:
            q.q4nx_kv_attention(c.cache, dev(qx), *args, ws=ws)
        if call in calls:
            with pytest.raises(q.Q4NXError) as e:
                q.q4nx_check(ws)
            assert e.value.status == q.Q4NX_E_INDEX, call
        q.q4nx_check(ws)                                   # reported once, and nothing else
    c.cache.pool.fill_(0xFF)
    c.fill().append_new()
    out = q.q4nx_kv_attention(c.cache, dev(qx), c.start, c.tlens, c.table, out_dtype="f32", ws=ws)
    assert torch.equal(out, good)
    assert np.isfinite(out.cpu().numpy()).all()
