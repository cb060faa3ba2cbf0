"""q4nx_logprobs on many rows of a full vocabulary, where a thread adds most elements.

Bounds.  A thread adds n <= ceil(V / 512) positive terms, each off by 2^-21, in binary32:
(n - 1) 2^-24 of the sum; its maximum moves at most once per 32 elements, each time by a
factor off by 2^-21; 16 more additions join the threads.  So z is within
    r = (n + 16) 2^-24 + (n / 32 + 2) 2^-21
of itself, lse within r + 2^-22 |lse|, a log-probability within 2^-22 |x| more, and the entropy, whose
second sum has the same steps, within 2 r (1 + sum p |x - m|).  Indexes: equal.
"""
import pytest
import torch

from test_gpu_logprobs import DEV, q  # noqa: F401  (q is a fixture)

pytestmark = pytest.mark.gpu
V = 151936


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 37, 64, 100, 152, 320])
@pytest.mark.parametrize("masked,flat", [(0, False), (19, False), (0, True)])
def test_full_vocabulary(q, M, dtype, masked, flat):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, V, generator=g, device=DEV) * (0.01 if flat else 3)
    if masked:
        x[:, 3::masked] = -float("inf")
    x = x.to(dtype)
    tokens = torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)
    got = q.q4nx_logprobs(x, tokens, top=20)
    n = -(-V // 512)
    r = (n + 16) * 2.0 ** -24 + (n / 32 + 2) * 2.0 ** -21
    value, idx = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(got.top_idx, idx[:, :20].to(torch.int32))
    d = x.double()
    lse = torch.logsumexp(d, 1)
    tol = r + 2.0 ** -22 * lse.abs()
    assert bool(((got.lse - lse).abs() <= tol).all())
    best = value[:, :20].double()
    assert bool(((got.top_logprob - (best - lse[:, None])).abs() <= tol[:, None] + 2.0 ** -22 * best.abs()).all())
    at = d.gather(1, tokens.long()[:, None])[:, 0]
    want, fin = at - lse, torch.isfinite(at)
    assert torch.equal(torch.isneginf(got.logprob), ~fin)
    assert bool(((got.logprob - want).abs() <= tol + 2.0 ** -22 * at.abs())[fin].all())
    m = d.amax(1, keepdim=True)
    p = torch.exp(d - lse[:, None])
    far = torch.where(p > 0, (m - d), 0.0)
    far = (p * far).sum(1)
    entropy = lse - m[:, 0] + far
    assert bool(((got.entropy - entropy).abs() <= 2 * r * (1 + far)).all())
