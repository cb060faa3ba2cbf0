"""The example of decode steps behind one prompt, operator by operator, against binary64.

Each operator is checked on the inputs it got (the previous operator's outputs), so that its own
bound holds: products (1e-3 + 2^-9) sum |w x| through the epilogue and 2^-8 of the value, attention over
the cached values 2^-11 + 2^-13 + 2^-20 of sum p |v| and 2^-8; the rotation is exact."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from test_gpu_kv import _bf16, _values
from test_gpu_rotary import kept, turn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    spec = importlib.util.spec_from_file_location("shared_prompt", os.path.join(ROOT, "examples", "shared_prompt.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod                       # dataclasses look their module up
    spec.loader.exec_module(mod)
    return mod


def _n(t):
    return t.double().cpu().numpy()


def _product(w, x):
    y, A = oracle.matmul(w.chunks.cpu().numpy(), w.kind, w.rows, w.cols, x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
    return y.reshape(len(x), -1), (1e-3 + 2.0 ** -9) * A.reshape(len(x), -1)


def _within(got, y, tol):
    tol = tol + 2.0 ** -23 * np.abs(y)                 # additions and products of the epilogue in binary32
    assert np.all(np.abs(_n(got).reshape(y.shape) - y) <= tol + 2.0 ** -8 * (np.abs(y) + tol))


def _attention(q, k, v, scale):
    """Output and sum p |v| of one row's heads: q [heads][dim], k, v [n][kv_heads][dim]."""
    y, A = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(len(q)):
        j = h // (len(q) // k.shape[1])
        l = k[:, j] @ q[h] * scale
        p = np.exp(l - l.max())
        p /= p.sum()
        y[h], A[h] = p @ v[:, j], p @ (2 * np.abs(v[:, j]) + np.abs(v[:, j]).max())
    return y, A


@pytest.mark.parametrize("count,prompt,encoder", [(5, 70, [3, 0, 40, 17, 64]), (33, 300, [20 + b for b in range(33)]), (3, 16, [1, 1, 1])])
def test_layer_by_operator(ex, count, prompt, encoder):
    s = ex.Sizes(hidden=512, inner=768, heads=8, kv_heads=2, head_dim=128, page_tokens=16, positions=400)
    layer = ex.Layer(s)
    reqs = ex.Requests(layer, count, prompt, 4, encoder)
    table, scale = layer.rotary.table.cpu().numpy(), s.head_dim ** -0.5
    full = torch.tensor(np.concatenate([[0], np.cumsum(encoder)]), dtype=torch.int32, device="cuda")
    ck, cv = (_n(t) for t in ex.q4.q4nx_kv_read(reqs.states, sum(encoder), full, reqs.states_lens, reqs.states_table, out_dtype="f32"))
    pk, pv = (_n(t) for t in ex.q4.q4nx_kv_read(reqs.cache, prompt, torch.tensor([0, prompt], dtype=torch.int32, device="cuda"), reqs.lens[:1],
                                                reqs.table[:1], out_dtype="f32"))
    x = torch.randn(count, s.hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    own_k, own_v = [], []
    for n in range(3):
        out = reqs.step(x)
        y, tol = _product(layer.qkv, x)
        _within(out["qkv"], y + _n(layer.bias), tol)
        qkv, pos = out["qkv"].float().cpu().numpy(), np.full(count, prompt + n)
        assert np.array_equal(out["turned"].float().cpu().numpy(), _bf16(turn(qkv[:, :s.heads], pos, table, False)))
        own_k.append(kept(turn(qkv[:, s.heads:s.heads + s.kv_heads], pos, table, False)).astype(np.float64))
        own_v.append(_values(qkv[:, s.heads + s.kv_heads:]).astype(np.float32).astype(np.float64))
        for b in range(count):
            kb, vb = np.concatenate([pk, *[k[b:b + 1] for k in own_k]]), np.concatenate([pv, *[v[b:b + 1] for v in own_v]])
            y, A = _attention(_n(out["turned"][b]), kb, vb, scale)
            _within(out["attention"][b], y, (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -20) * A)
            if encoder[b]:
                y, A = _attention(_n(out["cross_q"][b]), ck[int(full[b]):int(full[b + 1])], cv[int(full[b]):int(full[b + 1])], scale)
                _within(out["cross"][b], y, (2.0 ** -11 + 2.0 ** -13) * A)
            else:
                assert torch.all(out["cross"][b] == 0)
        y, tol = _product(layer.o, out["attention"].flatten(1))
        _within(out["h"], y + _n(x), tol)
        y, tol = _product(layer.c, out["h"])
        _within(out["cross_q"], y, tol)
        y, tol = _product(layer.d, out["cross"].flatten(1))
        _within(out["mid"], y + _n(out["h"]), tol)
        (g, tg), (u, tu) = _product(layer.gate, out["mid"]), _product(layer.up, out["mid"])
        tu = tu + 2.0 ** -8 * (np.abs(u) + tu)         # up's output is rounded
        act = g / (1 + np.exp(-g))
        ta = 1.13 * (tg + 2.0 ** -21 * np.abs(g)) + 2.0 ** -20 * np.abs(act)
        _within(out["gated"], act * u, ta * (np.abs(u) + tu) + np.abs(act) * tu)
        y, tol = _product(layer.down, out["gated"])
        _within(out["out"], y + _n(out["mid"]), tol)
        x = (out["out"].float() / out["out"].float().std()).bfloat16()
    assert reqs.lens.tolist() == [prompt + 3] * count
    ex.q4.q4nx_check(device="cuda:0")


def test_steps_captured_in_a_graph(ex):
    """A step as a graph, the lengths counted on the device: the same numbers as the calls one by one."""
    s = ex.Sizes(hidden=512, inner=768, heads=8, kv_heads=2, head_dim=64, page_tokens=16, positions=400)
    layer, outs = ex.Layer(s), []
    x = torch.randn(12, s.hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    for captured in (False, True):
        reqs = ex.Requests(layer, 12, 130, 8, [30] * 12)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = [reqs.step(x)["out"].clone()]
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    out = reqs.step(x)["out"]
            for _ in range(3):
                if captured:
                    graph.replay()
                    got.append(out.clone())
                else:
                    got.append(reqs.step(x)["out"].clone())
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        outs.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    ex.q4.q4nx_check(device="cuda:0")
