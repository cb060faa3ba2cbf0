"""The far negative tails of the activations: as long as a value is a normal number it keeps its bound.

x / (1 + exp(-z)) for z below -87: the denominator passes 2^126 and binary32's end, the value is 2^-126 and more until
SiLU's x = -91.9 and tanh GELU's x = -10.1.  Bound: 2^-20 of the value at a number within 2^-21 of the sum, which
moves it by 2^-21 (1 + |x| z'(x)) of itself; bf16 output half a step, 2^-8, more."""
import math

import numpy as np
import pytest
import torch

from test_gpu_epilogue import DEV, _f64, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu

SILU = [-60.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -89.5, -90.0, -90.5, -91.0, -91.5]
TANH = [-9.0, -9.5, -9.875, -9.9375, -10.0, -10.0625]


@pytest.mark.parametrize("M", [1, 2, 16, 64])
@pytest.mark.parametrize("act,points", [("silu", SILU), ("gelu_tanh", TANH)])
def test_tails(q, act, points, M):  # noqa: F811
    N, K = 64, 256
    W = q.Weight(torch.zeros(N // 32 * 5120, dtype=torch.uint8, device=DEV), q.Q4NX_Q4_1, N, K)
    X = torch.ones(M, K, device=DEV, dtype=torch.bfloat16)
    bias = torch.tensor((points * 16)[:N], device=DEV).bfloat16()    # the sum itself
    x = _f64(bias)
    assert set(x) == set(points)
    if act == "silu":
        z, slope = x, 1.0
    else:
        c = math.sqrt(2 / math.pi)
        z, slope = 2 * c * (x + 0.044715 * x ** 3), 2 * c * (1 + 3 * 0.044715 * x * x)
    v = x * np.exp(z) / (1 + np.exp(z))
    assert np.all(np.abs(v) >= 2.0 ** -126)
    tol = np.abs(v) * (2.0 ** -20 + 2.0 ** -21 * (1 + np.abs(x) * slope))
    for dt in ("f32", "bf16"):
        got = _f64(q.q4nx_gemm_epilogue(W, X, bias=bias, act=act, out_dtype=dt))
        t = tol + (2.0 ** -8 * (np.abs(v) + tol) if dt == "bf16" else 0)
        assert np.all(np.abs(got - v) <= t), (act, dt, x[np.argmax(np.abs(got - v)[0] - t)])
