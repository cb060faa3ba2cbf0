"""The serving operators, case by case: inputs, one call, a plain form and the formula in 64 bits.

One decode step of several requests, around the Q4NX products:

  append     new keys and values of each request go into its 4-bit paged cache, and are read back as the values kept
  attention  each request's query tokens attend to its cache
  lora       a Q4NX projection of up to 64 tokens, with each token's own low-rank adapter added
  logprobs   the lm_head logits' log-probabilities: the given token's, the entropy, the top alternatives

`own` False: elementary torch operations in 32 bits, rounded once at the end.
`own` True: the calls a user makes of the package.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases --

def listed():
    att = dict(op="attention", mixed=False, window=0)
    return [
        # the first answer tokens of one short chat: nothing but latency counts
        dict(att, name="attention short", batch=1, tokens=1, length=45, ragged=False, heads=16, kv_heads=8, dim=128, page=16),
        # a server's decode step: many requests of different lengths
        dict(att, name="attention decode batch", batch=48, tokens=1, length=6000, ragged=True, heads=32, kv_heads=8, dim=128, page=64),
        # one request over a very long document, odd length
        dict(att, name="attention long", batch=1, tokens=1, length=131071, ragged=False, heads=16, kv_heads=8, dim=128, page=256),
        # four drafted tokens of each request checked at once, wide heads, a sliding window that starts inside pages
        dict(att, name="attention drafts window", batch=16, tokens=4, length=9001, ragged=True, heads=16, kv_heads=4, dim=256, page=48, window=4097),
        # the next 64 tokens of a long prompt (the products' largest block) attend to what came before
        dict(att, name="attention prompt block", batch=1, tokens=64, length=16384, ragged=False, heads=32, kv_heads=8, dim=128, page=64),
        # a decode step's new token of every request
        dict(op="append", name="append decode", batch=48, tokens=1, length=6000, ragged=True, kv_heads=8, dim=128, page=64),
        # prompts of odd lengths that begin inside a page
        dict(op="append", name="append prompts", batch=3, tokens=1501, length=4001, ragged=True, kv_heads=8, dim=128, page=64),
        # one token of one request through a small projection with its adapter
        dict(op="lora", name="lora one token", kind="q4_1", tokens=1, rows=2048, cols=1024, rank=16, adapters=4, block=False),
        # 64 requests, nearly every one with an adapter of its own
        dict(op="lora", name="lora many requests", kind="q4_1", tokens=64, rows=12288, cols=4096, rank=16, adapters=64, block=False),
        # a 64-token prompt block of one request with one wide adapter, 8-bit weights
        dict(op="lora", name="lora prompt block", kind="q8_blk", tokens=64, rows=4096, cols=12288, rank=64, adapters=4, block=True),
        # one request's next token, with the alternatives that a client may ask for
        dict(op="logprobs", name="logprobs one row", rows=1, vocab=151936, top=20, dtype="f32"),
        # a 64-token block scored
        dict(op="logprobs", name="logprobs block", rows=64, vocab=151936, top=5, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "lora", "logprobs"])
    if op == "attention":
        dim, kv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        c = dict(op=op, dim=dim, kv_heads=kv, heads=kv * rng.choice([1, 2, 3, 4, 6, 8]), page=rng.choice([16, 48, 64, 256]),
                 batch=_log(rng, 1, 48), tokens=rng.choice([1, 1, 1, 2, 5, 17, 64]), ragged=rng.random() < 0.7)
        most = min(131072, 120_000_000 // (c["batch"] * kv * dim), 64 * 32 * 16384 // (c["batch"] * c["heads"] * c["tokens"]))
        c["length"] = _log(rng, c["tokens"], max(c["tokens"], most))
        c["window"] = _log(rng, 1, c["length"]) if rng.random() < 0.25 else 0
        c["mixed"] = c["tokens"] > 1 and rng.random() < 0.3
        return c
    if op == "append":
        dim, kv, batch = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 48)
        tokens = _log(rng, 1, max(1, 4500 * 1024 // (batch * dim * kv) if batch > 3 else 1500 * 1024 // (dim * kv)))
        return dict(op=op, batch=batch, tokens=tokens, length=tokens + _log(rng, 1, 2000) - 1, ragged=rng.random() < 0.7,
                    kv_heads=kv, dim=dim, page=rng.choice([16, 48, 64, 256]))
    if op == "lora":
        rows = 32 * _log(rng, 8, 384)
        cols = 256 * _log(rng, 1, max(1, 12288 * 4096 // (rows * 256) if rows > 4096 else 48))
        rank = rng.choice([8, 16, 16, 32, 64])
        return dict(op=op, kind=rng.choice(["q4_1", "q4_1", "q8_kr", "q8_blk"]), tokens=_log(rng, 1, 64), rows=rows, cols=cols,
                    rank=rank, adapters=_log(rng, 1, 1024 // rank), block=rng.random() < 0.4)
    return dict(op=op, rows=_log(rng, 1, 64), vocab=_log(rng, 1000, 151936), top=rng.choice([0, 1, 5, 20, 32]),
                dtype=rng.choice(["f32", "f32", "bf16"]))


def _lengths(c):
    """(cached tokens after the call, tokens of the call) of each request."""
    n, t = [], []
    for b in range(c["batch"]):
        share = 1.0 - 0.9 * math.fmod(b * 0.6180339887, 1.0) if c["ragged"] else 1.0
        tb = c["tokens"] if c["op"] != "append" or c["tokens"] == 1 else max(1, int(c["tokens"] * share))
        tb = 1 if c.get("mixed") and b else tb
        n.append(max(tb, int(c["length"] * share)))
        t.append(tb)
    return n, t


def _ids(c):
    """Each token's adapter, -1 for none."""
    n = c["adapters"]
    if c["block"]:
        return [n - 1] * c["tokens"]
    return [-1 if m % 9 == 8 else (7 * m + 3) % n for m in range(c["tokens"])]


def work(c):
    if c["op"] in ("attention", "append"):
        n, t = _lengths(c)
        per = c["kv_heads"] * c["dim"]
        if c["op"] == "append":       # 16-bit keys and values in, 5 bits a value kept, and read back in 32
            return {"bytes": sum(t) * per * 2 * (2 + 0.625 + 0.625 + 4), "flops": sum(t) * per * 2 * 6}
        seen = pairs = 0
        for nb, tb in zip(n, t):
            first = max(0, nb - tb + 1 - c["window"]) if c["window"] else 0
            seen += nb - first
            for i in range(tb):
                p = nb - tb + i + 1
                pairs += min(p, c["window"]) if c["window"] else p
        rows = sum(t) * c["heads"]
        return {"bytes": seen * per * 2 * 0.625 + rows * (c["dim"] * 4 + 4), "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "lora":
        used, m = len({i for i in _ids(c) if i >= 0}), c["tokens"]
        have = sum(i >= 0 for i in _ids(c))
        per = 0.625 if c["kind"] == "q4_1" else 1.0625
        side = c["rank"] * (c["rows"] + c["cols"])
        return {"bytes": c["rows"] * c["cols"] * per + used * side * 2 + 2 * m * (c["rows"] + c["cols"]),
                "flops": 2 * m * c["rows"] * c["cols"] + 2 * have * side}
    return {"bytes": c["rows"] * (c["vocab"] * (4 if c["dtype"] == "f32" else 2) + 16 + 8 * c["top"]), "flops": 6 * c["rows"] * c["vocab"]}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _start(t):
    return torch.tensor([0] + t, device=DEV).cumsum(0).to(torch.int32)


def _kv_inputs(c, seed):
    """The requests' lengths and page table, and all their keys and values: [cached tokens][kv_heads][dim] bf16."""
    g = _gen(seed)
    n, t = _lengths(c)
    need = [-(-v // c["page"]) for v in n]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    at, col = _start(need)[:-1].long()[:, None], torch.arange(max(need), device=DEV)[None]
    table = torch.where(col < torch.tensor(need, device=DEV)[:, None], perm[(at + col).clamp(max=pages - 1)], -1).to(torch.int32)
    shape = (sum(n), c["kv_heads"], c["dim"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    k[..., 5::37] *= 4                                     # a few channels are larger, as keys' are
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) + 0.25
    return dict(g=g, n=n, t=t, pages=pages, table=table, k=k, v=v, lens=torch.tensor(n, dtype=torch.int32, device=DEV), q_start=_start(t))


def _query(c, i):
    """The query tokens: the first part of a merged projection's output row."""
    width = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    merged = torch.randn(sum(i["t"]), width, generator=i["g"], device=DEV, dtype=torch.bfloat16)
    return merged[:, :c["heads"] * c["dim"]].unflatten(1, (c["heads"], c["dim"]))


def _new_rows(i):
    """Indexes of each request's last tokens among all cached ones."""
    end = torch.tensor(i["n"], device=DEV).cumsum(0)
    return torch.cat([torch.arange(int(e) - t, int(e), device=DEV) for e, t in zip(end.tolist(), i["t"])])


def _chunks(c, g):
    """Chunk bytes of a random weight."""
    n = c["rows"] // 32 * (c["cols"] // 256)
    codes = torch.randint(0, 256, (n, 4096 if c["kind"] == "q4_1" else 8192), generator=g, device=DEV, dtype=torch.uint8)
    if c["kind"] != "q4_1":
        codes = torch.where(codes == 128, 0, codes)        # int8 codes within -127..127
        return torch.cat([codes, (_normal(g, n, 256) * 0.005).abs().bfloat16().view(torch.uint8)], 1)
    s = (_normal(g, n, 256) * 0.02).abs() / 8
    z = -8 * s * (1 + 0.2 * (torch.rand(n, 256, generator=g, device=DEV) - 0.5))
    return torch.cat([codes, s.bfloat16().view(torch.uint8), z.bfloat16().view(torch.uint8)], 1)


def _lora_inputs(c, seed):
    g = _gen(seed)
    n, r = c["adapters"], c["rank"]
    return dict(chunks=_chunks(c, g).flatten(), x=_normal(g, c["tokens"], c["cols"]).bfloat16(),
                a=(_normal(g, n, r, c["cols"]) / math.sqrt(c["cols"])).bfloat16(), b=(_normal(g, n, c["rows"], r) * 0.05).bfloat16(),
                s=0.5 + torch.rand(n, generator=g, device=DEV), ids=torch.tensor(_ids(c), dtype=torch.int32, device=DEV))


def _logits_inputs(c, seed):
    g = _gen(seed)
    x = _normal(g, c["rows"], c["vocab"]) * 3
    hot = torch.randint(0, c["vocab"], (c["rows"], 8), generator=g, device=DEV)
    x.scatter_add_(1, hot, _normal(g, c["rows"], 8).abs() * 6)                       # a few likely tokens
    x[:, 3::19] = -math.inf                                                         # tokens that a grammar forbids
    x = x.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
    return dict(x=x, tokens=hot[:, 0].to(torch.int32).contiguous())


# ---------------------------------------------------------------- prepare --

def _quantise(x):
    """16-bit values to 4-bit codes, scale and middle of each 32, every step one operation in 32 bits."""
    v = x.float().unflatten(-1, (-1, 32))
    lo, hi = v.amin(-1), v.amax(-1)
    s = ((hi - lo) / 15).bfloat16()
    m = (lo + 8 * s.float()).bfloat16()
    step = s.float()[..., None]
    code = torch.where(step == 0, 0.0, torch.round((v - m.float()[..., None]) / torch.where(step == 0, 1.0, step)))
    return (code.clamp(-8, 7) + 8).to(torch.uint8).flatten(-2), s, m


def _plain_store(pool, at, x):
    """Codes two to a byte, scales and middles of new rows into a plain pool's rows `at`."""
    c, s, m = _quantise(x)
    pool["c"][at], pool["s"][at], pool["m"][at] = c[..., ::2] | c[..., 1::2] << 4, s, m


def _plain_load(pool, at):
    """The values of a plain pool's rows `at`, in 32 bits."""
    c = torch.stack([pool["c"][at] & 15, pool["c"][at] >> 4], -1).flatten(-2).float() - 8
    return (c.unflatten(-1, (-1, 32)) * pool["s"][at].float()[..., None] + pool["m"][at].float()[..., None]).flatten(-2)


def _plain_pool(c, pages):
    rows, h, d = pages * c["page"], c["kv_heads"], c["dim"]
    new = lambda w, t: torch.zeros(rows, h, w, dtype=t, device=DEV)  # noqa: E731
    return dict(c=new(d // 2, torch.uint8), s=new(d // 32, torch.bfloat16), m=new(d // 32, torch.bfloat16))


def _places(c, i, first, count):
    """Pool rows of positions first[b].. of each request, [batch][count]; where past its end, its last."""
    pos = (first[:, None] + torch.arange(count, device=DEV)[None]).clamp(min=0)
    pos = torch.minimum(pos, i["lens"].long()[:, None] - 1)
    return i["table"].long().gather(1, pos // c["page"]) * c["page"] + pos % c["page"]


def _filled(c, i, keep):
    """The cache as earlier calls left it, with each request's first keep[b] tokens in it."""
    rows = torch.cat([torch.arange(e - n, e - n + m, device=DEV) for e, n, m in zip(torch.tensor(i["n"]).cumsum(0).tolist(), i["n"], keep)])
    k, v = i["k"][rows], i["v"][rows]
    if own:
        # the cache lives in the layout of whoever reads it, so that each side fills its own
        import dequant_gemv_gb300 as q
        cache = q.KVCache.alloc(i["pages"], c["kv_heads"], c["dim"], c["page"], DEV)
        if sum(keep):
            q.q4nx_kv_append(cache, k, v, _start(keep), torch.tensor(keep, dtype=torch.int32, device=DEV), i["table"])
        return cache
    pools = _plain_pool(c, i["pages"]), _plain_pool(c, i["pages"])
    req = torch.repeat_interleave(torch.arange(len(keep), device=DEV), torch.tensor(keep, device=DEV))
    pos = torch.arange(len(rows), device=DEV) - _start(keep).long()[req]
    at = i["table"].long()[req, pos // c["page"]] * c["page"] + pos % c["page"]
    for pool, x in zip(pools, (k, v)):
        for j in range(0, len(rows), 1 << 16):
            _plain_store(pool, at[j:j + (1 << 16)], x[j:j + (1 << 16)])
    return pools


def prepare(c, seed):
    if c["op"] == "attention":
        i = _kv_inputs(c, seed)
        st = dict(q=_query(c, i), cache=_filled(c, i, i["n"]), scale=1 / math.sqrt(c["dim"]))
        return dict(st, c=c, most=(max(i["n"]), max(i["t"])), **{k: i[k] for k in ("lens", "q_start", "table")})
    if c["op"] == "append":
        i = _kv_inputs(c, seed)
        cache = _filled(c, i, [n - t for n, t in zip(i["n"], i["t"])])
        merged = torch.cat([i["k"][_new_rows(i)].flatten(1), i["v"][_new_rows(i)].flatten(1)], 1)    # one projection's output row
        k, v = (merged[:, j * c["kv_heads"] * c["dim"]:][:, :c["kv_heads"] * c["dim"]].unflatten(1, (c["kv_heads"], c["dim"])) for j in (0, 1))
        return dict(c=c, k=k, v=v, cache=cache, total=sum(i["t"]), **{k: i[k] for k in ("lens", "q_start", "table")})
    if c["op"] == "lora":
        i = _lora_inputs(c, seed)
        if own:
            import dequant_gemv_gb300 as q
            return dict(c=c, x=i["x"], ids=i["ids"], w=q.Weight(i["chunks"], q.KINDS[c["kind"]], c["rows"], c["cols"]),
                        adapters=q.Adapters(i["a"], i["b"], i["s"]))
        return dict(i, c=c)
    return dict(_logits_inputs(c, seed), c=c)


# -------------------------------------------------------------------- run --

def run(st):
    return (_run_own if own else _run_plain)[st["c"]["op"]](st)


def _own_attention(st):
    import dequant_gemv_gb300 as q
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    out = q.q4nx_kv_attention(st["cache"], st["q"], st["q_start"], st["lens"], st["table"], scale=st["scale"], window=st["c"]["window"], lse=lse)
    return out, lse


def _own_append(st):
    import dequant_gemv_gb300 as q
    q.q4nx_kv_append(st["cache"], st["k"], st["v"], st["q_start"], st["lens"], st["table"])
    return q.q4nx_kv_read(st["cache"], st["total"], st["q_start"], st["lens"], st["table"], out_dtype="f32")


def _own_lora(st):
    import dequant_gemv_gb300 as q
    return q.q4nx_gemm_lora(st["w"], st["x"], st["adapters"], st["ids"])


def _own_logprobs(st):
    import dequant_gemv_gb300 as q
    return tuple(q.q4nx_logprobs(st["x"], st["tokens"], top=st["c"]["top"]))


def _plain_attention(st):
    c, (most_n, most_t) = st["c"], st["most"]
    lens, start = st["lens"].long(), st["q_start"].long()
    t = start[1:] - start[:-1]
    first = (lens - t - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    span = min(most_n, c["window"] + most_t) if c["window"] else most_n
    at = _places(c, st, first, span)
    k, v = (_plain_load(pool, at) for pool in st["cache"])                           # [batch][span][kv_heads][dim]
    row = start[:-1, None] + torch.minimum(torch.arange(most_t, device=DEV)[None], t[:, None] - 1)
    q = st["q"][row].float().unflatten(2, (c["kv_heads"], -1))                       # [batch][tokens][kv_heads][group][dim]
    s = torch.einsum("bthgd,blhd->bhgtl", q, k) * st["scale"]
    key, pos = first[:, None] + torch.arange(span, device=DEV)[None], (lens - t)[:, None] + torch.arange(most_t, device=DEV)[None]
    see = key[:, None] <= pos[:, :, None]
    if c["window"]:
        see &= key[:, None] > pos[:, :, None] - c["window"]
    s = torch.where(see[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgtl,blhd->bthgd", p / z, v).flatten(2, 3)
    lse = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).flatten(2)
    req = torch.repeat_interleave(torch.arange(len(t), device=DEV), t, output_size=st["q"].shape[0])
    tok = torch.arange(st["q"].shape[0], device=DEV) - start[req]
    return o[req, tok].bfloat16(), lse[req, tok]


def _plain_append(st):
    c = st["c"]
    lens, start = st["lens"].long(), st["q_start"].long()
    t = start[1:] - start[:-1]
    req = torch.repeat_interleave(torch.arange(len(t), device=DEV), t, output_size=st["total"])
    pos = (lens - t)[req] + torch.arange(st["total"], device=DEV) - start[req]
    at = st["table"].long()[req, pos // c["page"]] * c["page"] + pos % c["page"]
    _plain_store(st["cache"][0], at, st["k"])
    _plain_store(st["cache"][1], at, st["v"])
    return _plain_load(st["cache"][0], at), _plain_load(st["cache"][1], at)


def _plain_weight(chunks, kind, rows, cols):
    """A weight's values in 32 bits, [rows][cols]."""
    b = chunks.view(rows // 32, cols // 256, -1)
    field = lambda o: b[..., o:o + 512].contiguous().view(torch.bfloat16).view(*b.shape[:2], 32, 8, 1).float()  # noqa: E731
    if kind == "q4_1":
        c = b[..., :4096].reshape(*b.shape[:2], 32, 8, 16)
        w = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() * field(4096) + field(4608)
    else:
        c = b[..., :8192].contiguous().view(torch.int8)
        if kind == "q8_kr":                                # code (r, k) at k*32 + r
            c = c.view(*b.shape[:2], 8, 32, 32).permute(0, 1, 4, 2, 3)
        else:                                              # at (r/16)*4096 + (k/32)*512 + (k%32)*16 + r%16
            c = c.view(*b.shape[:2], 2, 8, 32, 16).permute(0, 1, 2, 5, 3, 4).flatten(2, 3)
        w = c.float() * field(8192)
    return w.flatten(-2).permute(0, 2, 1, 3).reshape(rows, cols)


def _plain_lora(st):
    c = st["c"]
    x, i = st["x"].float(), st["ids"].long()
    y = x @ _plain_weight(st["chunks"], c["kind"], c["rows"], c["cols"]).T
    has, i = (i >= 0).float(), i.clamp(min=0)
    t = (st["a"].float()[i] @ x[:, :, None])               # [tokens][rank][1]
    add = (st["b"].float()[i] @ t)[..., 0]
    return (y + (has * st["s"][i])[:, None] * add).bfloat16()


def _plain_logprobs(st):
    x, top = st["x"].float(), st["c"]["top"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    lse = m + torch.log(z)
    entropy = torch.log(z)[:, 0] - (torch.where(e > 0, e * (x - m), 0.0).sum(1, keepdim=True) / z)[:, 0]
    value, idx = torch.sort(x, dim=1, descending=True, stable=True)
    return (x.gather(1, st["tokens"].long()[:, None]) - lse)[:, 0], entropy, lse[:, 0], idx[:, :top].to(torch.int32), value[:, :top] - lse


_run_own = dict(attention=_own_attention, append=_own_append, lora=_own_lora, logprobs=_own_logprobs)
_run_plain = dict(attention=_plain_attention, append=_plain_append, lora=_plain_lora, logprobs=_plain_logprobs)


# ------------------------------------------------------------------ exact --

def _kept(x):
    """What a 4-bit cache keeps of x, in 64 bits: codes, scales and middles by the rule, the values unrounded."""
    y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for g in range(x.shape[-1] // 32):
        part = x[..., 32 * g:32 * g + 32].float()
        lo = part.min(-1, keepdim=True).values
        s = ((part.max(-1, keepdim=True).values - lo) / 15.0).to(torch.bfloat16).float()
        mid = (lo + s * 8.0).to(torch.bfloat16).float()
        code = ((part - mid) / s).round().clamp(min=-8, max=7)
        code = torch.where(s > 0, code, torch.zeros_like(code))
        y[..., 32 * g:32 * g + 32] = code.double() * s.double() + mid.double()
    return y


def exact(c, seed):
    if c["op"] == "attention":
        i = _kv_inputs(c, seed)
        q, scale, w = _query(c, i), 1 / math.sqrt(c["dim"]), c["window"]
        outs, lses, end, begin = [], [], 0, 0
        for n, t in zip(i["n"], i["t"]):
            k, v = _kept(i["k"][end:end + n]), _kept(i["v"][end:end + n])
            qb = q[begin:begin + t].double()
            pos = torch.arange(n - t, n, device=DEV)[:, None]
            key = torch.arange(n, device=DEV)[None]
            hidden = (key > pos) | ((key <= pos - w) if w else torch.zeros_like(key > pos))
            group = c["heads"] // c["kv_heads"]
            o, l = torch.empty_like(qb), torch.empty(t, c["heads"], dtype=torch.float64, device=DEV)
            for h in range(c["heads"]):
                logits = (qb[:, h] @ k[:, h // group].T * scale).masked_fill(hidden, -math.inf)
                l[:, h] = torch.logsumexp(logits, 1)
                o[:, h] = torch.exp(logits - l[:, h:h + 1]) @ v[:, h // group]
            outs.append(o)
            lses.append(l)
            end, begin = end + n, begin + t
        return torch.cat(outs), torch.cat(lses)
    if c["op"] == "append":
        i = _kv_inputs(c, seed)
        rows = _new_rows(i)
        return _kept(i["k"][rows]), _kept(i["v"][rows])
    if c["op"] == "lora":
        i = _lora_inputs(c, seed)
        rows, cols = c["rows"], c["cols"]
        raw = i["chunks"].view(rows // 32 * (cols // 256), -1)
        w = torch.empty(rows, cols, dtype=torch.float64, device=DEV).view(rows // 32, 32, cols // 256, 256)
        r, k = torch.arange(32, device=DEV)[:, None], torch.arange(256, device=DEV)[None]
        head = 4096 if c["kind"] == "q4_1" else 8192
        for tc in range(cols // 256):
            chunk = raw[tc::cols // 256]
            scale = chunk[:, head:head + 512].contiguous().view(torch.bfloat16).double()[:, r * 8 + k // 32]
            if c["kind"] == "q4_1":
                code = (chunk[:, r * 128 + k // 2].int() >> (4 * (k % 2))) & 15
                zero = chunk[:, head + 512:].contiguous().view(torch.bfloat16).double()[:, r * 8 + k // 32]
                w[:, :, tc] = code.double() * scale + zero
            else:
                at = k * 32 + r if c["kind"] == "q8_kr" else r // 16 * 4096 + k // 32 * 512 + k % 32 * 16 + r % 16
                w[:, :, tc] = chunk[:, at].view(torch.int8).double() * scale
        y = i["x"].double() @ w.reshape(rows, cols).T
        for m, a in enumerate(_ids(c)):
            if a >= 0:
                y[m] += i["s"][a].double() * (i["b"][a].double() @ (i["a"][a].double() @ i["x"][m].double()))
        return y
    i = _logits_inputs(c, seed)
    x = i["x"].double()
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    entropy = -(p * torch.where(p > 0, x - lse[:, None], 0.0)).sum(1)
    best = torch.topk(x, max(1, c["top"]), dim=1).values[:, :c["top"]]
    return x[torch.arange(c["rows"], device=DEV), i["tokens"].long()] - lse, entropy, lse, None, best - lse[:, None]
