"""The example's decode step, operator by operator, against binary64.

Each operator is checked on the inputs it got (the previous operator's outputs), so
that its own bound holds: the products with adapters (1e-3 + 2^-9) sum |w x| and 2^-8 of the
value; attention over the cached values 2^-11 + 2^-13 of sum p |v| and 2^-8 of the value."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod                       # dataclasses look their module up
    spec.loader.exec_module(mod)
    return mod


def _n(t):
    return t.double().cpu().numpy()


def _product(w, x, ad, ids):
    y, A = oracle.matmul(w.chunks.cpu().numpy(), w.kind, w.rows, w.cols, x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
    y, A = y.reshape(len(x), -1).copy(), A.reshape(len(x), -1)
    a, b = _n(ad.a), _n(ad.b)
    S = np.zeros_like(y)
    for m, i in enumerate(ids):
        if i >= 0:
            y[m] += b[i] @ (a[i] @ _n(x[m]))
            S[m] = np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(_n(x[m])))
    return y, (1e-3 + 2.0 ** -9) * A + (w.cols + a.shape[1]) * 2.0 ** -23 * S


def _within(got, y, tol):
    assert np.all(np.abs(_n(got).reshape(y.shape) - y) <= tol + 2.0 ** -8 * (np.abs(y) + tol))


def test_step_by_step(ex):
    s = ex.Sizes(hidden=512, heads=8, kv_heads=2, head_dim=128, vocab=1024, page_tokens=16, rank=8)
    model = ex.Model(s)
    ids = [0, -1, 2, 1, 0]
    reqs = ex.Requests(model, 5, 70, ids)
    lengths = [1, 17, 64, 33, 50]
    reqs.prompt(lengths)
    tokens = torch.arange(5, device="cuda")
    for n in range(3):
        out = reqs.step(tokens)
        y, tol = _product(model.qkv, out["x"], model.qkv_adapters, ids)
        _within(out["qkv"], y, tol)
        assert reqs.lens.tolist() == [v + n + 1 for v in lengths]
        full = torch.tensor(np.concatenate([[0], np.cumsum(reqs.lens.tolist())]), dtype=torch.int32, device="cuda")
        k, v = ex.q4.q4nx_kv_read(reqs.cache, int(full[-1]), full, reqs.lens, reqs.table, out_dtype="f32")
        k, v, q = _n(k), _n(v), _n(out["qkv"][:, :s.heads])
        for b in range(5):
            kb, vb = k[int(full[b]):int(full[b + 1])], v[int(full[b]):int(full[b + 1])]
            # the newest token's cached values are its projection's, to half a step of 15 of its range
            new = _n(out["qkv"][b, s.heads:s.heads + s.kv_heads]).reshape(s.kv_heads, -1, 32)
            step = (new.max(-1) - new.min(-1))[..., None] / 15
            assert np.all(np.abs(kb[-1].reshape(new.shape) - new) <= 0.52 * step + 2.0 ** -7 * np.abs(new).max())
            for h in range(s.heads):
                l = kb[:, h // 4] @ q[b, h] * s.head_dim ** -0.5
                p = np.exp(l - l.max())
                p /= p.sum()
                got, want, A = _n(out["attention"][b, h]), p @ vb[:, h // 4], p @ (2 * np.abs(vb[:, h // 4]) + np.abs(vb).max())
                t = (2.0 ** -11 + 2.0 ** -13) * A
                assert np.all(np.abs(got - want) <= t + 2.0 ** -8 * (np.abs(want) + t))
        y, tol = _product(model.o, out["attention"].flatten(1), model.o_adapters, ids)
        h = _n(out["x"]) + y
        assert np.all(np.abs(_n(out["hidden"]) - h) <= 2 * (tol + 2.0 ** -8 * (np.abs(y) + np.abs(h) + tol)))
        x = _n(out["logits"])
        assert np.array_equal(out["tokens"].cpu().numpy(), x.argmax(1))
        lse = x.max(1) + np.log(np.exp(x - x.max(1, keepdims=True)).sum(1))
        assert np.all(np.abs(_n(out["logprobs"].top_logprob[:, 0]) - (x.max(1) - lse)) <= 2.0 ** -16 * (1 + np.abs(lse)))
        tokens = out["tokens"]
    ex.q4.q4nx_check(device="cuda:0")
