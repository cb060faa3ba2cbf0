"""The 4-bit key/value cache and its attention against the formulas in binary64.

Bounds.  Cached values: exact (the rule is a chain of single binary32 operations).
Attention, binary32 output: each weight p*scale is rounded to fp16, 2^-11 of
itself, so an output moves by at most 2^-11 of A = sum p (|(code-8) scale| +
|mid|) / sum p; a logit's binary32 sum (terms up to 136 |q| scale, 256
channels) is off by less than 2^-14, which moves p by 2^-13 of itself in all.
bf16 output: half an ulp, 2^-8 of the value, more.  lse: 2^-13 + 2^-20 |lse|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    import dequant_gemv_gb300

    return dequant_gemv_gb300


def _bf16(x):
    """binary32 -> the nearest bf16, as binary32 (ties to even)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return b.view(np.float32)


def _quantize(x):
    """(code - 8, scale, mid) of bf16 values [..., D] by the rule, in binary32 steps."""
    v = x.astype(np.float32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        lo, hi = v.min(-1), v.max(-1)
        s = _bf16((hi - lo) / np.float32(15))
        m = _bf16(lo + np.float32(8) * s)
        c = np.clip(np.rint((v - m[..., None]) / s[..., None]), -8, 7)
        c = np.where(s[..., None] == 0, 0, c)
        bad = ~np.isfinite(v).all(-1) | ~np.isfinite(s) | ~np.isfinite(m)
    s, m = np.where(bad, np.nan, s), np.where(bad, np.nan, m)
    return np.nan_to_num(c).astype(np.float64), s.astype(np.float64), m.astype(np.float64)


def _values(x):
    c, s, m = _quantize(x)
    return (c * s[..., None] + m[..., None]).reshape(x.shape)


class Case:
    """Requests with their tokens: `lens` cached tokens, the last `new` of them in the call."""

    def __init__(self, q, lens, new, kv, dim, page, seed=0, spare=2, fill=0xFF, extra_tokens=0):
        self.q, self.lens, self.new, self.kv, self.dim, self.page = q, lens, new, kv, dim, page
        self.rng = np.random.default_rng([seed, dim, kv, page, len(lens)])
        need = [max(1, -(-n // page)) for n in lens]
        pages = sum(need) + spare
        perm = self.rng.permutation(pages)
        table = np.full((len(lens), max(need) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.cache = q.KVCache.alloc(pages, kv, dim, page, DEV)
        self.cache.pool.fill_(fill)                     # what a page held before: NaN patterns
        self.table = torch.from_numpy(table).to(DEV)
        self.tlens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        self.tokens = int(sum(new)) + extra_tokens
        self.k = [self.draw(n) for n in lens]           # per request [len][kv][dim], bf16 values
        self.v = [self.draw(n) + np.float32(0.25) for n in lens]
        self.v = [_bf16(x) for x in self.v]

    def draw(self, n, heads=None):
        x = self.rng.normal(size=(n, heads or self.kv, self.dim)).astype(np.float32)
        x[..., 5::37] *= 4
        return _bf16(x)

    def fill(self):
        """Everything but the call's tokens, as earlier calls left it."""
        old = [n - t for n, t in zip(self.lens, self.new)]
        old = [max(0, o) for o in old]
        self.append(self.stack(self.k, 0, old), self.stack(self.v, 0, old), old, old)
        return self

    def stack(self, xs, lo, hi):
        parts = [x[(lo if isinstance(lo, int) else lo[b]):hi[b]] for b, x in enumerate(xs)]
        return np.concatenate(parts) if parts else np.zeros((0, self.kv, self.dim), np.float32)

    def append(self, k, v, new, lens):
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        self.q.q4nx_kv_append(self.cache, dev(k), dev(v), start, torch.tensor(lens, dtype=torch.int32, device=DEV), self.table)

    def append_new(self):
        """The call's tokens: those of positions below 0 are noise that must not be kept."""
        ks, vs = [], []
        for b, (n, t) in enumerate(zip(self.lens, self.new)):
            miss = max(0, t - n)
            ks += [self.draw(miss), self.k[b][max(0, n - t):]]
            vs += [self.draw(miss), self.v[b][max(0, n - t):]]
        self.append(np.concatenate(ks), np.concatenate(vs), self.new, self.lens)
        return self


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(torch.bfloat16)


def exact(c, qx, scale, window, heads):
    """(out, lse, A) in binary64."""
    outs = np.zeros((c.tokens, heads, c.dim))
    lse = np.full((c.tokens, heads), -np.inf)
    A = np.zeros_like(outs)
    g, at = heads // c.kv, 0
    for b, (n, t) in enumerate(zip(c.lens, c.new)):
        k = _values(c.k[b]).astype(np.float64)
        cv, sv, mv = _quantize(c.v[b])
        v = (cv * sv[..., None] + mv[..., None]).reshape(c.v[b].shape)
        va = (np.abs(cv * sv[..., None]) + np.abs(mv[..., None])).reshape(c.v[b].shape)
        for j in range(t):
            pos = n - t + j
            lo = max(0, pos - window + 1) if window else 0
            if pos >= 0:
                for h in range(heads):
                    l = k[lo:pos + 1, h // g] @ qx[at + j, h].astype(np.float64) * scale
                    m = l.max()
                    p = np.exp(l - m)
                    lse[at + j, h] = m + np.log(p.sum())
                    outs[at + j, h] = p @ v[lo:pos + 1, h // g] / p.sum()
                    A[at + j, h] = p @ va[lo:pos + 1, h // g] / p.sum()
        at += t
    return outs, lse, A


def check(c, qx, out, lse, scale, window, heads, rows=None):
    y, l, A = exact(c, qx, scale, window, heads)
    n = int(sum(c.new)) if rows is None else rows
    y, l, A = y[:n], l[:n], A[:n]
    got, gl = out[:n].float().cpu().numpy().astype(np.float64), lse[:n].cpu().numpy().astype(np.float64)
    tol = (2.0 ** -11 + 2.0 ** -13) * A
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
    empty = np.isinf(l)
    assert np.array_equal(np.isneginf(gl), empty) and not np.isnan(got).any()
    assert np.all(got[empty] == 0)
    assert np.all(np.abs(got - y) <= tol), np.max((np.abs(got - y) - tol))
    assert np.all(np.abs(gl - l)[~empty] <= 2.0 ** -13 + 2.0 ** -20 * np.abs(l[~empty]))


def attend(c, heads, window=0, scale=None, out_dtype="f32", merged=True):
    scale = c.dim ** -0.5 if scale is None else scale
    qx = c.draw(c.tokens, heads)
    row = np.concatenate([qx.reshape(c.tokens, -1), c.draw(c.tokens, 2 * c.kv).reshape(c.tokens, -1)], 1) if merged else qx.reshape(c.tokens, -1)
    qt = dev(row)[:, :heads * c.dim].unflatten(1, (heads, c.dim))
    lse = torch.full((c.tokens, heads), 7.0, device=DEV)
    out = c.q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, c.table, scale=scale, window=window, out_dtype=out_dtype, lse=lse)
    return qx, out, lse, scale


# ------------------------------------------------------------ append, read --

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,page", [(1, 16), (3, 48), (8, 64)])
def test_append_keeps_the_rule_exactly(q, dim, kv, page):
    c = Case(q, [1, 15, 16, 17, 70, 0, 130], [1, 15, 3, 17, 5, 0, 130], kv, dim, page).fill().append_new()
    for dt in ("f32", "bf16"):
        k, v = q.q4nx_kv_read(c.cache, c.tokens, c.start, c.tlens, c.table, out_dtype=dt)
        for got, xs in ((k, c.k), (v, c.v)):
            want = _values(c.stack(xs, [n - t for n, t in zip(c.lens, c.new)], c.lens)).astype(np.float32)
            want = _bf16(want) if dt == "bf16" else want
            assert np.array_equal(got.float().cpu().numpy(), want)
    # and every token of every request, those of earlier calls among them
    k, v = q.q4nx_kv_read(c.cache, sum(c.lens), torch.tensor(np.concatenate([[0], np.cumsum(c.lens)]), dtype=torch.int32, device=DEV),
                          c.tlens, c.table, out_dtype="f32")
    assert np.array_equal(k.cpu().numpy(), _values(np.concatenate(c.k)).astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), _values(np.concatenate(c.v)).astype(np.float32))
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_writes_only_its_tokens(q, dim):
    c = Case(q, [40, 33], [1, 2], 2, dim, 16, fill=0x5A)
    before = c.cache.pool.clone()
    c.append_new()
    changed = int((c.cache.pool != before).sum())
    assert 0 < changed <= 3 * 2 * 2 * (dim // 2 + dim // 8)
    c.append_new()                                         # the same again: same bytes
    assert int((c.cache.pool != before).sum()) == changed


def test_append_of_special_groups(q):
    c = Case(q, [6], [6], 1, 64, 16)
    k = c.k[0]
    k[0, 0, :32] = 1.5                                     # constant: scale 0, the value itself
    k[1, 0, 3] = np.inf
    k[2, 0, 40] = np.nan
    k[3, 0, 0], k[3, 0, 1] = 3e38, -3e38                   # a range beyond binary32
    k[4, 0, :] = 0
    k[5, 0, :32] = _bf16(np.arange(32, dtype=np.float32) * np.float32(2.0 ** -130))
    c.k[0] = _bf16(k) if np.isfinite(k).all() else k
    c.append_new()
    got = q.q4nx_kv_read(c.cache, 6, c.start, c.tlens, c.table, out_dtype="f32")[0].cpu().numpy()
    assert np.array_equal(got, _values(c.k[0]).astype(np.float32), equal_nan=True)
    assert np.isnan(got[1, 0, :32]).all() and np.isnan(got[2, 0, 32:]).all() and np.isnan(got[3, 0, :32]).all()
    assert not np.isnan(got[1, 0, 32:]).any() and not np.isnan(got[2, 0, :32]).any() and np.all(got[0, 0, :32] == 1.5)


def test_tokens_before_the_start_and_of_no_request(q):
    # request 0 has more tokens than its length; the call has two tokens of no request
    c = Case(q, [2, 20], [5, 1], 2, 64, 16).fill().append_new()
    k, _ = q.q4nx_kv_read(c.cache, 8, c.start, c.tlens, c.table, out_dtype="f32")
    k = k.cpu().numpy()
    assert np.all(k[:3] == 0) and np.all(k[6:] == 0)
    assert np.array_equal(k[3:5], _values(c.k[0]).astype(np.float32))
    c.tokens = 8
    qx, out, lse, scale = attend(c, 4)
    check(c, qx, out, lse, scale, 0, 4)


# --------------------------------------------------------------- attention --

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,group,page,new", [(1, 1, 16, 1), (2, 4, 64, 1), (4, 8, 48, 1), (2, 3, 16, 1), (1, 16, 32, 1), (2, 2, 64, 4),
                                               (1, 7, 16, 5), (2, 8, 48, 9), (1, 4, 64, 64)])
def test_attention_matches(q, dim, kv, group, page, new):
    lens = [max(new, n) for n in (1, 2, 15, 16, 17, 33, 250, 1025)]
    c = Case(q, lens, [new] * len(lens), kv, dim, page, seed=group).fill().append_new()
    for dt in ("f32", "bf16"):
        qx, out, lse, scale = attend(c, kv * group, out_dtype=dt)
        check(c, qx, out, lse, scale, 0, kv * group)
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("dim,window", [(64, 1), (128, 16), (128, 17), (256, 100), (64, 1000), (128, 5000)])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_attention_window(q, dim, window, new):
    lens = [max(new, n) for n in (5, 16, 100, 129, 2000)]
    c = Case(q, lens, [new] * 5, 2, dim, 48, seed=window).fill().append_new()
    qx, out, lse, scale = attend(c, 6, window=window)
    check(c, qx, out, lse, scale, window, 6)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 63 - 1])
@pytest.mark.parametrize("new", [9, 100])
def test_attention_window_beyond_every_length(q, window, new):
    # a window that hides nothing, rows before the first position among them
    c = Case(q, [1, 3, 500], [new, new, new], 2, 128, 16, seed=new).fill().append_new()
    qx, out, lse, scale = attend(c, 8, window=window)
    check(c, qx, out, lse, scale, 0, 8)
    q.q4nx_check(device=DEV)


def test_attention_mixed_empty_and_short_requests(q):
    # no tokens in the call; an empty cache; rows before the first position; one long split request
    c = Case(q, [40, 0, 3, 9000, 1, 64], [0, 2, 7, 3, 1, 64], 2, 128, 64).fill().append_new()
    for heads in (2, 10):
        qx, out, lse, scale = attend(c, heads)
        check(c, qx, out, lse, scale, 0, heads)
    qx, out, lse, scale = attend(c, 4, window=33)
    check(c, qx, out, lse, scale, 33, 4)
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("dim,group,new", [(128, 2, 1), (64, 8, 1), (256, 4, 3), (128, 4, 20)])
def test_attention_one_long_request_split_between_ctas(q, dim, group, new):
    c = Case(q, [20011], [new], 1, dim, 256).fill().append_new()
    qx, out, lse, scale = attend(c, group)
    check(c, qx, out, lse, scale, 0, group)
    again = attend(Same(c, qx), group)
    assert torch.equal(out, again[1]) and torch.equal(lse, again[2])       # fixed order of the sums


class Same:
    """The same case with the queries given."""

    def __init__(self, c, qx):
        self.__dict__.update(c.__dict__)
        self.c, self.qx = c, qx

    def draw(self, n, heads=None):
        return self.qx if heads == self.qx.shape[1] and n == len(self.qx) else self.c.draw(n, heads)


def test_attention_many_requests(q):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 300, 1024)]
    c = Case(q, lens, [1] * 1024, 1, 64, 16).fill().append_new()
    qx, out, lse, scale = attend(c, 2)
    check(c, qx, out, lse, scale, 0, 2)


def test_attention_sharp_and_scaled_values(q):
    # logits far apart, keys and values of very different sizes from token to token
    c = Case(q, [700, 90], [1, 2], 2, 128, 64)
    for b in range(2):
        f = np.exp2(c.rng.integers(-20, 21, size=(c.lens[b], c.kv, 1))).astype(np.float32)
        c.v[b] = _bf16(c.v[b] * f)
        c.k[b] = _bf16(c.k[b] * np.exp2(c.rng.integers(-3, 3, size=(c.lens[b], c.kv, 1))).astype(np.float32))
    c.fill().append_new()
    for scale in (0.5, -0.3, 1e-3, 0.0):
        qx, out, lse, scale = attend(c, 4, scale=scale)
        y, l, A = exact(c, qx, scale, 0, 4)
        # logits up to some hundreds: their binary32 sums are off by up to 2^-17 of sum |q k| times scale
        got = out.float().cpu().numpy().astype(np.float64)
        big = abs(scale) * max(np.abs(qx).sum(-1).max() * np.abs(np.concatenate(c.k)).max(), 1.0)
        tol = (2.0 ** -11 + 2.0 ** -13 + 2 * 2.0 ** -17 * big) * A
        assert np.all(np.abs(got - y) <= tol)
        assert np.all(np.abs(lse.cpu().numpy() - l) <= 2.0 ** -13 + 2.0 ** -17 * big)


def test_attention_nan_stays_where_it_is_seen(q):
    c = Case(q, [50, 50], [4, 1], 1, 64, 16)
    c.k[0][48, 0, 3] = np.nan                             # seen by the last two of four tokens
    c.v[0][49, 0, 40] = np.inf                            # seen by the last token only, in one group
    c.fill().append_new()
    qx, out, lse, scale = attend(c, 2)
    got, l = out.cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(got[:2]).all() and np.isfinite(l[:2]).all() and np.isnan(got[2:4]).all() and np.isnan(l[2:4]).all()
    assert np.isfinite(got[4]).all()
    c.k[0][48, 0, 3] = 0.5
    c.fill().append_new()
    qx, out, lse, scale = attend(c, 2)
    got = out.cpu().numpy()
    assert np.isfinite(got[:3]).all() and np.isfinite(got[3, :, :32]).all() and np.isnan(got[3, :, 32:]).all()


# Many rows per request (more than 64 on average, 64 or 128 channels) go to a kernel
# of 256-row units of two tiles, on the tensor cores; 256 channels stay where they are.
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,new,window", [(4, 100, 0), (3, 50, 0), (1, 129, 70), (3, 100, 70), (16, 33, 1), (5, 60, 64), (1, 300, 257)])
def test_attention_many_rows(q, dim, group, new, window):
    lens = [new, new + 1, max(1, new - 30), 333, 1025]     # the third has rows before its first position
    c = Case(q, lens, [new] * len(lens), 2, dim, 48, seed=new + group).fill().append_new()
    for dt in ("f32", "bf16"):
        qx, out, lse, scale = attend(c, 2 * group, window=window, out_dtype=dt)
        check(c, qx, out, lse, scale, window, 2 * group)


def test_attention_many_rows_of_some_requests(q):
    # the average decides: requests of 600 rows, of one token, of none, and an empty cache
    c = Case(q, [40, 0, 3, 9000, 1, 700], [0, 2, 7, 3, 1, 300], 2, 128, 64).fill().append_new()
    qx, out, lse, scale = attend(c, 4)
    check(c, qx, out, lse, scale, 0, 4)
    again = attend(Same(c, qx), 4)
    assert torch.equal(out, again[1]) and torch.equal(lse, again[2])


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_many_rows_nan_stays_where_it_is_seen(q, dim):
    c = Case(q, [400, 90], [200, 70], 1, dim, 16)
    c.k[0][300, 0, 3] = np.nan                            # seen by the tokens from position 300 on
    c.v[0][260, 0, 40] = np.inf                           # from position 260 on, in one group
    c.fill().append_new()
    qx, out, lse, scale = attend(c, 2)
    got, l = out.cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(l[:100]).all() and np.isnan(l[100:200]).all() and np.isnan(got[100:200]).all()
    assert np.isfinite(got[:60]).all() and np.isfinite(got[200:]).all() and np.isfinite(l[200:]).all()
    assert np.isfinite(got[60:100, :, :32]).all() and np.isnan(got[60:100, :, 32:64]).all() and np.isfinite(got[60:100, :, 64:]).all()
    # a window past them: those rows are finite again, and right
    qx, out, lse, scale = attend(c, 2, window=20)
    got = out.cpu().numpy()
    assert np.isfinite(got[120:]).all() and np.isfinite(got[80:100]).all() and np.isfinite(lse.cpu().numpy()[120:]).all()


def test_attention_many_rows_sharp_and_scaled_values(q):
    c = Case(q, [700, 90], [130, 70], 2, 128, 64)
    for b in range(2):
        f = np.exp2(c.rng.integers(-20, 21, size=(c.lens[b], c.kv, 1))).astype(np.float32)
        c.v[b] = _bf16(c.v[b] * f)
        c.k[b] = _bf16(c.k[b] * np.exp2(c.rng.integers(-3, 3, size=(c.lens[b], c.kv, 1))).astype(np.float32))
    c.fill().append_new()
    for scale in (0.5, -0.3, 1e-3, 0.0):
        qx, out, lse, scale = attend(c, 4, scale=scale)
        y, l, A = exact(c, qx, scale, 0, 4)
        # as for few rows; a key is kept to 2^-17 of itself
        got = out.float().cpu().numpy().astype(np.float64)
        big = abs(scale) * max(np.abs(qx).sum(-1).max() * np.abs(np.concatenate(c.k)).max(), 1.0)
        tol = (2.0 ** -11 + 2.0 ** -13 + 2 * 2.0 ** -16 * big) * A
        assert np.all(np.abs(got - y) <= tol)
        assert np.all(np.abs(lse.cpu().numpy() - l) <= 2.0 ** -13 + 2.0 ** -16 * big)


def test_attention_many_rows_in_a_graph_and_bad_indexes(q):
    c = Case(q, [300, 200], [80, 90], 2, 128, 64).fill().append_new()
    qx, out, lse, scale = attend(c, 4)
    qt, out2 = dev(qx), torch.zeros_like(out)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, c.table, out=out2, out_dtype="f32", ws=ws)
    for _ in range(3):
        g.replay()
    assert torch.equal(out, out2)
    for i, x in (((0, 1), 10 ** 6), ((1, 0), -1)):
        table = c.table.clone()
        table[i] = x
        q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, table, ws=ws)
        with pytest.raises(q.Q4NXError) as e:
            q.q4nx_check(ws)
        assert e.value.status == q.Q4NX_E_INDEX
    g.replay()
    assert torch.equal(out, out2)


def test_attention_on_another_stream_and_in_a_graph(q):
    c = Case(q, [300, 20], [1, 1], 2, 128, 64).fill().append_new()
    qx, out, lse, scale = attend(c, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, out2, lse2, _ = attend(Same(c, qx), 4)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    qt, out3 = dev(qx), torch.zeros_like(out)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.q4nx_kv_attention(c.cache, qt, c.start, c.tlens, c.table, out=out3, out_dtype="f32", ws=ws)
    for _ in range(3):
        g.replay()
    assert torch.equal(out, out3)


def test_pool_beyond_32_bit_offsets(q):
    page = q.q4nx_kv_page_bytes(128, 8, 64)
    pages = (5 << 30) // page
    c = Case(q, [100], [2], 8, 128, 64)
    c.cache = q.KVCache.alloc(pages, 8, 128, 64, DEV)
    c.table = torch.tensor([[pages - 1, (1 << 32) // page, -1]], dtype=torch.int32, device=DEV)
    c.fill().append_new()
    k, _ = q.q4nx_kv_read(c.cache, 2, c.start, c.tlens, c.table, out_dtype="f32")
    assert np.array_equal(k.cpu().numpy(), _values(c.k[0][98:]).astype(np.float32))
    qx, out, lse, scale = attend(c, 8)
    check(c, qx, out, lse, scale, 0, 8)


def test_bad_indexes_are_reported_and_the_workspace_stays_usable(q):
    c = Case(q, [40, 30], [1, 1], 2, 64, 16).fill().append_new()
    qx, good, _, scale = attend(c, 4)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    bad = []
    for name, b, i, x in (("table", 0, 1, 10 ** 6), ("table", 0, 2, -1), ("lens", 0, None, -3), ("lens", 0, None, 10 ** 6),
                          ("start", 1, None, 5), ("start", 0, None, -1)):
        t = {"table": c.table.clone(), "lens": c.tlens.clone(), "start": c.start.clone()}
        if i is None:
            t[name][b] = x
        else:
            t[name][b, i] = x
        bad.append(t)
    for t in bad:
        for call in ("append", "read", "attention"):
            if call == "append":
                if t["table"][0, 1] != c.table[0, 1]:
                    continue                               # the new token's own page is a good one
                q.q4nx_kv_append(c.cache, dev(c.draw(2)), dev(c.draw(2)), t["start"], t["lens"], t["table"], ws=ws)
            elif call == "read":
                if t["table"][0, 1] != c.table[0, 1]:
                    continue
                q.q4nx_kv_read(c.cache, 2, t["start"], t["lens"], t["table"], ws=ws)
            else:
                q.q4nx_kv_attention(c.cache, dev(qx), t["start"], t["lens"], t["table"], ws=ws)
            if call != "attention" and (t["start"] != c.start).any():
                continue                                   # tokens of no request: nothing to report
            with pytest.raises(q.Q4NXError) as e:
                q.q4nx_check(ws)
            assert e.value.status == q.Q4NX_E_INDEX, (call, t)
    q.q4nx_check(ws)
    c.fill().append_new()
    out = q.q4nx_kv_attention(c.cache, dev(qx), c.start, c.tlens, c.table, out_dtype="f32", ws=ws)
    assert torch.equal(out, good)


@pytest.mark.parametrize("lens,new,kv", [([40, 30, 20], [1, 1, 0], 2), ([80] * 39, [80] * 38 + [0], 4)])
def test_bad_requests_without_tokens_are_reported(q, lens, new, kv):
    # a range out of order, a length of a request that has no tokens, in the first
    # 32 requests and beyond: append (by tokens, by blocks) and read report them and serve the others
    c = Case(q, lens, new, kv, 64, 16).fill().append_new()
    want = q.q4nx_kv_read(c.cache, c.tokens, c.start, c.tlens, c.table, out_dtype="f32")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    k, v = (dev(np.concatenate([x[n - t:] for x, n, t in zip(xs, lens, new)])) for xs in (c.k, c.v))
    for name, x in (("start", -1), ("start", 0), ("lens", -1), ("lens", 10 ** 6)):
        t = {"start": c.start.clone(), "lens": c.tlens.clone()}
        t[name][-1] = x
        c.cache.pool.fill_(0xFF)
        c.fill()
        for call in ("append", "read"):
            if call == "append":
                q.q4nx_kv_append(c.cache, k, v, t["start"], t["lens"], c.table, ws=ws)
            else:
                got = q.q4nx_kv_read(c.cache, c.tokens, t["start"], t["lens"], c.table, out_dtype="f32", ws=ws)
            with pytest.raises(q.Q4NXError) as e:
                q.q4nx_check(ws)
            assert e.value.status == q.Q4NX_E_INDEX, (call, name, x)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses(q):
    c = Case(q, [40], [1], 2, 64, 16)
    x = dev(c.draw(1))
    for k, v, start, lens, table in (
            (x, x[:, :1], c.start, c.tlens, c.table), (x.float(), x, c.start, c.tlens, c.table),
            (x, x, c.start.long(), c.tlens, c.table), (x, x, c.start[:1], c.tlens, c.table),
            (x, x, c.start, c.tlens, c.table.cpu()), (x[..., ::2], x[..., ::2], c.start, c.tlens, c.table),
            (x.transpose(1, 2), x.transpose(1, 2), c.start, c.tlens, c.table)):
        with pytest.raises(ValueError):
            q.q4nx_kv_append(c.cache, k, v, start, lens, table)
    with pytest.raises(ValueError):
        q.q4nx_kv_attention(c.cache, x, c.start, c.tlens, c.table, lse=torch.zeros(1, 3, device=DEV))
    with pytest.raises(ValueError):
        q.q4nx_kv_attention(c.cache, x, c.start, c.tlens, c.table, out=torch.zeros(1, 2, 64, device=DEV))
    with pytest.raises(q.Q4NXError) as e:
        q.q4nx_kv_attention(c.cache, dev(c.draw(1, 3)), c.start, c.tlens, c.table)
    assert e.value.status == q.Q4NX_E_SHAPE
    # no tokens at all: an empty answer
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert q.q4nx_kv_attention(c.cache, x[:0], none, c.tlens, c.table).shape == (0, 2, 64)
