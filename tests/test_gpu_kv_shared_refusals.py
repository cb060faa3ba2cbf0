"""What q4nx_kv_attention_shared leaves of a call with bad numbers in it, through the C entry point.

The rows of requests that are refused (and of tokens of no request) stay as they were, outputs
and log-sums, whatever the scratch held before; those of the other requests are what they are without them, within
the bounds of tests/test_gpu_kv_shared.py.  Both orders of the two passes: few rows a group (the prefixes first), many
rows a group and few a request (the prefixes second), many of both.

refused() is the rule as the header has it, restated on the host."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, dev, exact, q  # noqa: F401  (q is a fixture)
from test_gpu_kv_shared import Shared

pytestmark = pytest.mark.gpu

# prefixes of whole pages, in the tables of all requests: a group that begins elsewhere finds the same positions
FORMS = {"few": [(48, [(2, 1), (20, 1)]), (64, [(1, 1), (4, 1)])],
         "crowd": [(48, [(2, 1), (20, 1)] * 24), (64, [(1, 1), (4, 1)])],
         "long": [(2000, [(2, 1), (20, 1)] * 24), (1600, [(1, 1), (4, 1)])],          # prefixes that are cut between CTAs
         "prompts": [(48, [(65, 65), (70, 66)]), (64, [(70, 70), (66, 66)])]}


def refused(first, shared, start, lens, tokens, cap):
    """Which requests are."""
    out = []
    for b, n in enumerate(lens):
        T = start[b + 1] - start[b]
        ok = 0 <= start[b] <= start[b + 1] <= tokens and 0 <= n <= cap
        at = [g for g in range(len(shared)) if first[g] <= b < first[g + 1] and first[g] >= max(first[:g], default=0)]
        ok = ok and len(at) > 0
        if ok:
            s, f0, f1 = shared[at[0]], first[at[0]], first[at[0] + 1]
            ok = 0 <= s <= cap and 0 <= f0 and f1 <= len(lens) and 0 <= start[f0] <= start[f1] <= tokens and (T == 0 or start[f0] <= start[b] and start[b + 1] <= start[f1]) and (T == 0 or s == 0 or n - T >= s)
        out.append(not ok)
    return out


class Call:
    def __init__(self, q, form, dim, heads=8):  # noqa: F811
        self.c = c = Shared(q, FORMS[form] if isinstance(form, str) else form, 2, dim, 16, hidden=False).fill().append_new()
        self.heads, self.ws = heads, torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
        self.qx = c.draw(c.tokens, heads)
        self.qt = dev(self.qx)
        self.y, self.l, self.A = exact(c, self.qx, dim ** -0.5, 0, heads)
        self.t = dict(first=c.first, shared=c.shared, start=c.start, lens=c.tlens)

    def run(self, f32, **bad):
        """(out, lse) of the call with some of its numbers others; scratch, out and lse hold something else before."""
        c, q, t = self.c, self.c.q, dict(self.t, **bad)  # noqa: F841
        L, by = q.lib, ctypes.byref
        out = torch.full((c.tokens, self.heads, c.dim), 5.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
        lse = torch.full((c.tokens, self.heads), 7.0, device=DEV)
        scratch = torch.full((L.q4nx_kv_attention_shared_scratch(by(c.cache.c()), c.tokens, self.heads),), 0xFF, dtype=torch.uint8, device=DEV)
        b = q.q4nx_kv_batch(t["start"].data_ptr(), t["lens"].data_ptr(), c.table.data_ptr(), len(c.lens), c.table.shape[1], c.tokens)
        g = q.q4nx_kv_groups(t["first"].data_ptr(), t["shared"].data_ptr(), t["shared"].numel(), 0)
        st = L.q4nx_kv_attention_shared(by(c.cache.c()), by(b), by(g), self.qt.data_ptr(), self.heads * c.dim, self.heads, c.dim ** -0.5, out.data_ptr(),
                                        int(f32), lse.data_ptr(), self.ws.data_ptr(), self.ws.numel(), scratch.data_ptr(), scratch.numel(),
                                        torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, written):
        """The rows of `written` tokens are right, the others as they were."""
        rest = ~written
        assert torch.all(out[torch.from_numpy(rest)] == 5) and torch.all(lse[torch.from_numpy(rest)] == 7)
        got, gl = out.double().cpu().numpy()[written], lse.double().cpu().numpy()[written]
        y, l, A = self.y[written], self.l[written], self.A[written]
        tol = (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -20) * A
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
        assert np.all(np.abs(got - y) <= tol)
        assert np.all(np.abs(gl - l) <= 2.0 ** -13 + 2.0 ** -20 * np.abs(l))

    def bad(self, f32, **bad):
        c, q, t = self.c, self.c.q, {k: v.tolist() for k, v in dict(self.t, **bad).items()}  # noqa: F841
        no = refused(t["first"], t["shared"], t["start"], t["lens"], c.tokens, c.table.shape[1] * c.page)
        written = np.zeros(c.tokens, bool)
        for b, r in enumerate(no):
            if not r:
                written[t["start"][b]:t["start"][b + 1]] = True
        assert not written.all()                                   # something of it is refused
        good = self.run(f32)
        self.check(*self.run(f32, **bad), written)
        # the report still stands: a sound call beside it is what it was
        again = self.run(f32)
        assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
        with pytest.raises(q.Q4NXError) as e:
            q.q4nx_check(self.ws)
        assert e.value.status == q.Q4NX_E_INDEX
        q.q4nx_check(self.ws)

    def changed(self, name, at, x):
        t = self.t[name].clone()
        t[at] = x
        return {name: t}


# a request: of a group's first, of others; a group: what it shares, its bounds, its tokens
BAD = [("lens", 0, -1), ("lens", 1, 10 ** 6), ("lens", 1, 48), ("lens", 2, -7), ("lens", -1, 3), ("shared", 0, -1), ("shared", 0, 10 ** 6),
       ("shared", 1, 10 ** 6), ("first", -1, 10 ** 6), ("first", -1, 0), ("first", 1, -3), ("first", 0, 1), ("first", 0, -1),
       ("start", 0, -4), ("start", 1, 10 ** 6), ("start", 2, 10 ** 6), ("start", -1, 10 ** 6), ("start", -1, 0)]


@pytest.mark.parametrize("name,at,x", BAD)
@pytest.mark.parametrize("form,dim", [("few", 64), ("few", 256), ("crowd", 64), ("crowd", 128), ("crowd", 256), ("long", 128), ("long", 256), ("prompts", 128), ("prompts", 256)])
def test_refused_rows_stay_as_they_were(q, form, dim, name, at, x):  # noqa: F811
    call = Call(q, form, dim)
    for f32 in (True, False):
        call.bad(f32, **call.changed(name, at, x))


@pytest.mark.parametrize("name,at,x", [("first", 0, -1), ("first", 0, -2 ** 31), ("first", 2, 10 ** 6), ("first", -1, 10 ** 6), ("start", 3, -1), ("shared", 1, -1)])
@pytest.mark.parametrize("many", [1, 16])
def test_groups_that_share_nothing(q, many, name, at, x):  # noqa: F811
    """Refused like the others where their bounds or tokens are out of range."""
    call = Call(q, [(0, [(40, many)] * 3), (0, [(33, 1), (5, 5)]), (48, [(40, many)] * 3)], 128)
    call.bad(True, **call.changed(name, at, x))


@pytest.mark.parametrize("dim", [128, 256])
def test_tokens_of_no_request_inside_a_group(q, dim):  # noqa: F811
    """Ranges of two requests out of order: their tokens belong to no request, those around them do."""
    call = Call(q, "crowd", dim)
    call.bad(True, **call.changed("start", 5, -1))


@pytest.mark.parametrize("form,dim", [("few", 64), ("crowd", 128), ("prompts", 256)])
def test_requests_outside_their_groups_tokens(q, form, dim):  # noqa: F811
    """The last bound before some requests' tokens: the other pass has no part of them."""
    forms = {"few": [(48, [(5, 1)] * 4)] * 2, "crowd": [(48, [(5, 1)] * 40)] * 2, "prompts": [(48, [(70, 66)] * 4)] * 2}
    call = Call(q, forms[form], dim)
    call.bad(True, **call.changed("start", -1, int(call.c.start[-1]) - (2 if form != "prompts" else 70)))


@pytest.mark.parametrize("form", ["few", "crowd"])
@pytest.mark.parametrize("first", [[0, 4, 2, 6, 8], [0, 2, 10 ** 6, 6, 8], [0, 5, 4, 8, 8], [2, 1, 4, 6, 8], [0, 2, 4, -6, 8]])
def test_groups_out_of_order(q, form, first):  # noqa: F811
    """Groups that overlap those before them are refused; the ones before are not."""
    each = [(2, 1), (20, 1)] if form == "few" else [(2, 13), (20, 13)]
    call = Call(q, [(48, [(13 + n, t) for n, t in each]) for _ in range(4)], 128)
    # all groups share the same positions: a request may be in any of them
    call.c.table[:, :3] = call.c.table[0, :3]
    for b in range(8):
        call.c.k[b][:48], call.c.v[b][:48] = call.c.k[0][:48], call.c.v[0][:48]
    call.y, call.l, call.A = exact(call.c, call.qx, 128 ** -0.5, 0, 8)
    call.bad(True, first=torch.tensor(first, dtype=torch.int32, device=DEV))


def test_one_group_of_many_out_of_order(q):  # noqa: F811
    call = Call(q, [(16 * (1 + g % 3), [(2, 1), (5, 1)]) for g in range(40)], 64)
    for g, x in ((20, 37), (33, 10 ** 6), (1, -1)):
        call.bad(True, **call.changed("first", g, x))
