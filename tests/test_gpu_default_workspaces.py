"""The binding's default workspaces around captured graphs: one made during a capture is
ready for calls before the first replay and not the graph's to reset, and one that a
larger call has replaced stays the graph's."""
import torch
import pytest

from test_gpu_kv import DEV, Case, attend, check, dev, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu


def fresh_stream(q):  # noqa: F811
    """A stream for which no workspace has been made."""
    for _ in range(64):
        s = torch.cuda.Stream()
        if not any(key[2] == s.cuda_stream for key in q._ws):
            return s
    pytest.fail("every stream has a workspace")


def kv_workspace(q, s):  # noqa: F811
    return q._ws[("kv", torch.device(DEV).index, s.cuda_stream)]


def captured(c, s, qt):
    """The case's attention in a graph captured on stream s, with the default workspace."""
    out = torch.full((c.tokens, qt.shape[1], c.dim), 7.0, device=DEV)
    lse = torch.full((c.tokens, qt.shape[1]), 7.0, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        c.q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, c.table, out=out, out_dtype="f32", lse=lse)
    return g, out, lse


@pytest.mark.parametrize("new,heads", [(1, 4), (100, 4)])
def test_first_call_of_a_stream_inside_a_capture(q, new, heads):  # noqa: F811
    # units cut between CTAs: their parts are counted in the workspace
    c = Case(q, [20011], [new], 1, 128, 256, seed=new).fill().append_new()
    qx, want, wlse, scale = attend(c, heads, merged=False)
    if new == 1:
        check(c, qx, want, wlse, scale, 0, heads)
    qt, s = dev(qx), fresh_stream(q)
    g, out, lse = captured(c, s, qt)
    with torch.cuda.stream(s):
        ws = kv_workspace(q, s)
        assert int(torch.count_nonzero(ws)) == 0            # before any replay
        early = q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, c.table, out_dtype="f32")
        assert torch.equal(early, want)
        for _ in range(3):
            g.replay()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        # an error that is not yet read survives a replay
        bad = c.tlens.clone()
        bad[0] = -1
        q.q4nx_kv_attention(c.cache, qt, c.start, bad, c.table)
        g.replay()
        with pytest.raises(q.Q4NXError) as e:
            q.q4nx_check(device=DEV)
        assert e.value.status == q.Q4NX_E_INDEX
        q.q4nx_check(device=DEV)
    s.synchronize()


@pytest.mark.parametrize("new,heads", [(1, 4), (100, 4)])
def test_a_graph_keeps_a_workspace_that_became_too_small(q, new, heads):  # noqa: F811
    small = Case(q, [20011], [new], 1, 64, 256, seed=new).fill().append_new()
    large = Case(q, [5000], [1], 1, 128, 64).fill().append_new()
    qx, want, wlse, scale = attend(small, heads, merged=False)
    qt, s = dev(qx), fresh_stream(q)
    with torch.cuda.stream(s):
        attend(small, heads)
        size = kv_workspace(q, s).numel()
        g, out, lse = captured(small, s, qt)
        qx2, got, glse, scale2 = attend(large, 2)           # needs more
        assert kv_workspace(q, s).numel() > size
        check(large, qx2, got, glse, scale2, 0, 2)
        # whatever takes the memory that is free now
        taken = [torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(4)]
        for _ in range(3):
            g.replay()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert all(int((t != 0x5A).sum()) == 0 for t in taken)
        again = attend(large, 2)
        check(large, *again[:3], again[3], 0, 2)
        # the graph's errors are found in the workspace that it kept
        small.tlens.fill_(-1)
        g.replay()
        with pytest.raises(q.Q4NXError) as e:
            q.q4nx_check(device=DEV)
        assert e.value.status == q.Q4NX_E_INDEX
        q.q4nx_check(device=DEV)
    s.synchronize()


def test_workspaces_of_the_products_inside_a_capture(q):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(1)
    chunks = torch.randint(0, 100, (8 * 4 * 8704,), generator=g, device=DEV, dtype=torch.uint8)
    chunks.view(-1, 8704)[:, 8192:] = torch.full((8 * 4, 256), 0.01, device=DEV).bfloat16().view(torch.uint8)
    w = q.Weight(chunks, q.Q4NX_Q8_KR, 256, 1024)
    X = torch.randn(64, 1024, generator=g, device=DEV).bfloat16()
    want1, want64 = q.q4nx_gemv(w, X[0]), q.q4nx_gemm_m64(w, X)
    s, graph = fresh_stream(q), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        y1, y64 = q.q4nx_gemv(w, X[0]), q.q4nx_gemm_m64(w, X)
    with torch.cuda.stream(s):
        assert torch.equal(q.q4nx_gemv(w, X[0]), want1) and torch.equal(q.q4nx_gemm_m64(w, X), want64)
        graph.replay()
        assert torch.equal(y1, want1) and torch.equal(y64, want64)
        q.q4nx_check(device=DEV)
    s.synchronize()
