"""More serving operators, case by case: inputs, one call, a plain form and the formula in 64 bits.

What a decode or prompt step of several requests needs around the 4-bit cache and the Q4NX products:

  rotary     new queries and keys are turned by their positions on the way into the cache, which is read back
  shared     attention of a batch whose requests share a long prefix, each with tokens of its own after it
  cross      attention to cached states of another sequence, of another length, all of them seen
  product    a Q4NX projection of up to 64 tokens with bias, activation, gate and residual in its epilogue

`own` False: elementary torch operations in 32 bits, rounded once at the end.
`own` True: the calls a user makes of the package.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases --

def listed():
    shared = dict(op="shared", ragged=True)
    cross = dict(op="cross")
    return [
        # a few answers to one short chat, sampled at once: latency
        dict(shared, name="shared short", batch=4, groups=1, tokens=1, shared=300, length=45, heads=16, kv_heads=8, dim=128, page=16),
        # a server's decode step behind one system prompt that ends inside a page
        dict(shared, name="shared system prompt", batch=48, groups=1, tokens=1, shared=8191, length=600, heads=32, kv_heads=8, dim=128, page=64),
        # drafted tokens of requests about two documents, wide heads
        dict(shared, name="shared drafts", batch=12, groups=2, tokens=4, shared=16001, length=500, heads=16, kv_heads=4, dim=256, page=48),
        # many answers about one very long document
        dict(shared, name="shared long", batch=16, groups=1, tokens=1, shared=65537, length=1000, heads=32, kv_heads=8, dim=128, page=256),
        # the next token of one transcript: as many kv heads as heads
        dict(cross, name="cross one token", batch=1, tokens=1, length=1500, ragged=False, heads=16, kv_heads=16, dim=64, page=16),
        # a batch that looks at images or documents of different sizes
        dict(cross, name="cross batch", batch=32, tokens=1, length=4097, ragged=True, heads=32, kv_heads=8, dim=128, page=64),
        # prompts of the answering side
        dict(cross, name="cross prompts", batch=4, tokens=449, length=6000, ragged=True, heads=32, kv_heads=8, dim=128, page=64),
        # a decode step's new token of every request, far into their texts
        dict(op="rotary", name="rotary decode", batch=48, tokens=1, length=131000, ragged=True, heads=32, kv_heads=8, dim=128, page=64, turned=128, pairs=False),
        # prompts of odd lengths that begin inside a page
        dict(op="rotary", name="rotary prompts", batch=3, tokens=1501, length=4001, ragged=True, heads=32, kv_heads=8, dim=128, page=64, turned=128, pairs=False),
        # one token back into the residual stream
        dict(op="product", name="product one token", kind="q4_1", tokens=1, rows=1024, cols=2048, act="none", bias=False, mul=False, residual=True),
        # a 64-token block's gate, activated and multiplied by the other half
        dict(op="product", name="product gate", kind="q4_1", tokens=64, rows=12288, cols=4096, act="silu", bias=False, mul=True, residual=False),
        # 33 requests through 8-bit weights with everything on
        dict(op="product", name="product biased", kind="q8_blk", tokens=33, rows=4096, cols=12288, act="gelu_tanh", bias=True, mul=False, residual=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "shared", "shared", "cross", "product"])
    if op == "product":
        rows = 32 * _log(rng, 8, 384)
        cols = 256 * _log(rng, 1, max(1, 12288 * 4096 // (rows * 256) if rows > 4096 else 48))
        return dict(op=op, kind=rng.choice(["q4_1", "q4_1", "q8_kr", "q8_blk"]), tokens=_log(rng, 1, 64), rows=rows, cols=cols,
                    act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.5,
                    mul=rng.random() < 0.4, residual=rng.random() < 0.5)
    dim, kv, page = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([16, 48, 64, 256])
    c = dict(op=op, dim=dim, kv_heads=kv, heads=kv * rng.choice([1, 2, 3, 4, 6, 8]), page=page, batch=_log(rng, 1, 48), ragged=rng.random() < 0.7)
    if op == "rotary":
        c["tokens"] = _log(rng, 1, max(1, 4500 * 5120 // (c["batch"] * dim * (c["heads"] + kv))))
        c["length"] = c["tokens"] + _log(rng, 1, 131072) - 1
        c["turned"] = dim // rng.choice([1, 1, 2, 4])
        c["pairs"] = rng.random() < 0.3
        return c
    c["tokens"] = rng.choice([1, 1, 1, 2, 5, 17, 64])
    most = min(65536, 300_000_000 // (c["batch"] * kv * dim), 13_000_000_000 // (c["batch"] * c["heads"] * c["tokens"] * dim))
    c["length"] = _log(rng, 1, max(1, most))
    if op == "shared":
        c["length"] = c["tokens"] + _log(rng, 1, max(1, most // 4)) - 1
        c["shared"] = _log(rng, 1, max(1, most - c["length"]))
        c["groups"] = rng.randint(1, min(3, c["batch"]))
    return c


def _share(c, b):
    return 1.0 - 0.9 * math.fmod(b * 0.6180339887, 1.0) if c["ragged"] else 1.0


def _groups(c):
    """(first request, shared tokens) of each group; the first requests' list ends with the batch."""
    first = [c["batch"] * g // c["groups"] for g in range(c["groups"] + 1)]
    return first, [max(1, int(c["shared"] * (1 - 0.3 * g))) for g in range(c["groups"])]


def _prefix(c):
    """Tokens that each request shares with its group."""
    first, length = _groups(c)
    return [length[g] for g in range(c["groups"]) for _ in range(first[g], first[g + 1])]


def _lengths(c):
    """(cached tokens, tokens of the call) of each request."""
    n, t = [], []
    for b in range(c["batch"]):
        tb = c["tokens"]
        if c["op"] == "rotary" and tb > 1:
            tb = max(1, int(tb * _share(c, b)))
        nb = max(1 if c["op"] == "cross" else tb, int(c["length"] * _share(c, b)))
        n.append(nb)
        t.append(tb)
    if c["op"] == "shared":
        n = [a + b for a, b in zip(n, _prefix(c))]
    return n, t


def work(c):
    if c["op"] == "product":
        m, per = c["tokens"], 0.625 if c["kind"] == "q4_1" else 1.0625
        each = 2 * m * c["rows"]                            # what the epilogue reads and writes, 16 bits each
        return {"bytes": c["rows"] * c["cols"] * per + 2 * m * c["cols"] + each * (1 + c["mul"] + c["residual"]) + 2 * c["rows"] * c["bias"],
                "flops": 2 * m * c["rows"] * c["cols"]}
    n, t = _lengths(c)
    per, width = c["kv_heads"] * c["dim"], c["heads"] * c["dim"]
    if c["op"] == "rotary":       # 16-bit queries in and out, keys and values in, 5 bits a value kept, and read back in 32
        return {"bytes": sum(t) * (width * 4 + per * 2 * (2 + 0.625 + 0.625 + 4)), "flops": sum(t) * (width * 3 + per * 2 * 6)}
    seen = sum(n) - (sum(_prefix(c)) - sum(_groups(c)[1]) if c["op"] == "shared" else 0)      # a shared token is read once
    pairs = 0
    for nb, tb in zip(n, t):
        pairs += tb * nb if c["op"] == "cross" else sum(nb - tb + i + 1 for i in range(tb))
    return {"bytes": seen * per * 2 * 0.625 + sum(t) * c["heads"] * (c["dim"] * 4 + 4), "flops": 4 * pairs * width}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _start(t):
    return torch.tensor([0] + t, device=DEV).cumsum(0).to(torch.int32)


def _kv(c, g, tokens):
    """Keys and values of cached tokens: [tokens][kv_heads][dim] bf16."""
    shape = (tokens, c["kv_heads"], c["dim"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    k[..., 5::37] *= 4                                     # a few channels are larger, as keys' are
    return k, torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) + 0.25


def _cache_inputs(c, seed):
    """The requests' lengths and pages, and their keys and values as (position range, k, v) parts of each request.

    A shared prefix's whole pages stand in the tables of all requests of the group; where it ends
    inside a page, every request has that page for itself, the prefix's last tokens in it."""
    g = _gen(seed)
    n, t = _lengths(c)
    page, batch = c["page"], c["batch"]
    first, length = _groups(c) if c["op"] == "shared" else ([0, batch], [0])
    need = [-(-v // page) for v in n]
    have = [[0] * v for v in need]                         # each request's pages, numbered as they are handed out
    fill = []                                              # each request's first position that is filled through its own table
    pages = 0
    for b in range(batch):
        grp = max(i for i in range(len(length)) if first[i] <= b)
        lead, whole = first[grp], length[grp] // page
        for j in range(need[b]):
            if b != lead and j < whole:
                have[b][j] = have[lead][j]
            else:
                have[b][j], pages = pages, pages + 1
        fill.append(0 if b == lead else whole * page)
    pages += 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    rows = torch.tensor([h + [-1] * (max(need) - len(h)) for h in have], device=DEV)
    table = torch.where(rows >= 0, perm[rows.clamp(min=0)], -1).to(torch.int32)
    prefix = [_kv(c, g, s) for s in length]
    own_k, own_v = _kv(c, g, sum(n) - (sum(_prefix(c)) if c["op"] == "shared" else 0))
    parts, at = [], 0
    for b in range(batch):
        grp = max(i for i in range(len(length)) if first[i] <= b)
        m = n[b] - length[grp]
        parts.append((prefix[grp], (own_k[at:at + m], own_v[at:at + m])))
        at += m
    return dict(g=g, n=n, t=t, pages=pages, table=table, parts=parts, fill=fill, first=_ints(first), shared=_ints(length),
                lens=_ints(n), q_start=_start(t))


def _rotary_inputs(c, seed):
    """New tokens of every request: merged rows of queries, keys and values, pages for the new positions alone, cosines and sines."""
    g = _gen(seed)
    n, t = _lengths(c)
    page = c["page"]
    span = [(nb - tb) // page for nb, tb in zip(n, t)]
    need = [-(-nb // page) - s for nb, s in zip(n, span)]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["batch"], max(-(-nb // page) for nb in n)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, (s, m) in enumerate(zip(span, need)):
        table[b, s:s + m] = perm[at:at + m]
        at += m
    merged = torch.randn(sum(t), (c["heads"] + 2 * c["kv_heads"]) * c["dim"], generator=g, device=DEV, dtype=torch.bfloat16)
    half = c["turned"] // 2
    angle = torch.arange(max(n), dtype=torch.float64, device=DEV)[:, None] * 1e6 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    turns = torch.stack([angle.cos(), angle.sin()], -1).float()           # as a server keeps them, [positions][pairs][2]
    x = merged.unflatten(1, (-1, c["dim"]))
    return dict(q=x[:, :c["heads"]], k=x[:, c["heads"]:c["heads"] + c["kv_heads"]], v=x[:, c["heads"] + c["kv_heads"]:], n=n, t=t,
                pages=pages, table=table, turns=turns, lens=_ints(n), q_start=_start(t))


def _query(c, i):
    """The query tokens: the first part of a merged projection's output row."""
    width = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    merged = torch.randn(sum(i["t"]), width, generator=i["g"], device=DEV, dtype=torch.bfloat16)
    return merged[:, :c["heads"] * c["dim"]].unflatten(1, (c["heads"], c["dim"]))


def _chunks(c, g):
    """Chunk bytes of a random weight."""
    n = c["rows"] // 32 * (c["cols"] // 256)
    codes = torch.randint(0, 256, (n, 4096 if c["kind"] == "q4_1" else 8192), generator=g, device=DEV, dtype=torch.uint8)
    if c["kind"] != "q4_1":
        codes = torch.where(codes == 128, 0, codes)        # int8 codes within -127..127
        return torch.cat([codes, (_normal(g, n, 256) * 0.0003).abs().bfloat16().view(torch.uint8)], 1)
    s = (_normal(g, n, 256) * 0.02).abs() / 8
    z = -8 * s * (1 + 0.2 * (torch.rand(n, 256, generator=g, device=DEV) - 0.5))
    return torch.cat([codes, s.bfloat16().view(torch.uint8), z.bfloat16().view(torch.uint8)], 1)


def _product_inputs(c, seed):
    g = _gen(seed)
    side = lambda on, *shape: _normal(g, *shape).bfloat16() if on else None  # noqa: E731
    return dict(chunks=_chunks(c, g).flatten(), x=_normal(g, c["tokens"], c["cols"]).bfloat16(), bias=side(c["bias"], c["rows"]),
                mul=side(c["mul"], c["tokens"], c["rows"]), residual=side(c["residual"], c["tokens"], c["rows"]))


# ---------------------------------------------------------------- prepare --

def _quantise(x):
    """Values in 32 bits to 4-bit codes, scale and middle of each 32, every step one operation in 32 bits."""
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


def _filled(c, i):
    """The cache as earlier calls left it: every prefix once, then each request's own tokens."""
    if own:
        # the cache lives in the layout of whoever reads it, so that each side fills its own
        import dequant_gemv_gb300 as q
        cache = q.KVCache.alloc(i["pages"], c["kv_heads"], c["dim"], c["page"], DEV)
    else:
        pools = _plain_pool(c, i["pages"]), _plain_pool(c, i["pages"])
    for b, (n, f, parts) in enumerate(zip(i["n"], i["fill"], i["parts"])):
        k, v = (torch.cat([parts[0][w][f:], parts[1][w]]) for w in (0, 1))
        if own:
            q.q4nx_kv_append(cache, k, v, _start([n - f]), i["lens"][b:b + 1], i["table"][b:b + 1])
            continue
        pos = torch.arange(f, n, device=DEV)
        at = i["table"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]
        for pool, x in zip(pools, (k, v)):
            _plain_store(pool, at, x)
    return cache if own else pools


def prepare(c, seed):
    if c["op"] in ("shared", "cross"):
        i = _cache_inputs(c, seed)
        st = dict(q=_query(c, i), cache=_filled(c, i), scale=1 / math.sqrt(c["dim"]))
        return dict(st, c=c, most=(max(i["n"]), max(i["t"])), **{k: i[k] for k in ("lens", "q_start", "table", "first", "shared")})
    if c["op"] == "rotary":
        i = _rotary_inputs(c, seed)
        if own:
            import dequant_gemv_gb300 as q
            keep = dict(cache=q.KVCache.alloc(i["pages"], c["kv_heads"], c["dim"], c["page"], DEV), rotary=q.Rotary(i["turns"], interleaved=c["pairs"]))
        else:
            keep = dict(cache=(_plain_pool(c, i["pages"]), _plain_pool(c, i["pages"])), turns=i["turns"])
        return dict(keep, c=c, total=sum(i["t"]), **{k: i[k] for k in ("q", "k", "v", "lens", "q_start", "table")})
    i = _product_inputs(c, seed)
    if own:
        import dequant_gemv_gb300 as q
        i["w"] = q.Weight(i.pop("chunks"), q.KINDS[c["kind"]], c["rows"], c["cols"])
    return dict(i, c=c)


# -------------------------------------------------------------------- run --

def run(st):
    return (_run_own if own else _run_plain)[st["c"]["op"]](st)


def _own_shared(st):
    import dequant_gemv_gb300 as q
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    out = q.q4nx_kv_attention_shared(st["cache"], st["q"], st["q_start"], st["lens"], st["table"], st["first"], st["shared"],
                                     scale=st["scale"], lse=lse)
    return out, lse


def _own_cross(st):
    import dequant_gemv_gb300 as q
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    out = q.q4nx_kv_attention_cross(st["cache"], st["q"], st["q_start"], st["lens"], st["table"], scale=st["scale"], lse=lse)
    return out, lse


def _own_rotary(st):
    import dequant_gemv_gb300 as q
    turned = q.q4nx_kv_append_rotary(st["cache"], st["rotary"], st["q"], st["k"], st["v"], st["q_start"], st["lens"], st["table"])
    return turned, *q.q4nx_kv_read(st["cache"], st["total"], st["q_start"], st["lens"], st["table"], out_dtype="f32")


def _own_product(st):
    import dequant_gemv_gb300 as q
    return q.q4nx_gemm_epilogue(st["w"], st["x"], bias=st["bias"], act=st["c"]["act"], mul=st["mul"], residual=st["residual"])


def _plain_attention(st):
    c, (most_n, most_t) = st["c"], st["most"]
    lens, start = st["lens"].long(), st["q_start"].long()
    t = start[1:] - start[:-1]
    key = torch.arange(most_n, device=DEV)[None]
    place = torch.minimum(key, (lens - 1)[:, None])
    at = st["table"].long().gather(1, place // c["page"]) * c["page"] + place % c["page"]
    k, v = (_plain_load(pool, at) for pool in st["cache"])                           # [batch][length][kv_heads][dim]
    row = start[:-1, None] + torch.minimum(torch.arange(most_t, device=DEV)[None], t[:, None] - 1)
    q = st["q"][row].float().unflatten(2, (c["kv_heads"], -1))                       # [batch][tokens][kv_heads][group][dim]
    s = torch.einsum("bthgd,blhd->bhgtl", q, k) * st["scale"]
    last = (lens - t)[:, None] + torch.arange(most_t, device=DEV)[None] if c["op"] == "shared" else (lens - 1)[:, None].expand(-1, most_t)
    s = torch.where((key[:, None] <= last[:, :, None])[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgtl,blhd->bthgd", p / z, v).flatten(2, 3)
    lse = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).flatten(2)
    req = torch.repeat_interleave(torch.arange(len(t), device=DEV), t, output_size=st["q"].shape[0])
    tok = torch.arange(st["q"].shape[0], device=DEV) - start[req]
    return o[req, tok].bfloat16(), lse[req, tok]


def _turn(x, cs, turned, pairs):
    """Rows [tokens][heads][dim] turned by their tokens' cosines and sines, every step one operation in 32 bits."""
    x, rest = x.float()[..., :turned], x.float()[..., turned:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (x[..., ::2], x[..., 1::2]) if pairs else (x[..., :turned // 2], x[..., turned // 2:])
    y = (a * c - b * s), (b * c + a * s)
    return torch.cat([torch.stack(y, -1).flatten(-2) if pairs else torch.cat(y, -1), rest], -1)


def _plain_rotary(st):
    c = st["c"]
    lens, start = st["lens"].long(), st["q_start"].long()
    t = start[1:] - start[:-1]
    req = torch.repeat_interleave(torch.arange(len(t), device=DEV), t, output_size=st["total"])
    pos = (lens - t)[req] + torch.arange(st["total"], device=DEV) - start[req]
    at = st["table"].long()[req, pos // c["page"]] * c["page"] + pos % c["page"]
    cs = st["turns"][pos]
    _plain_store(st["cache"][0], at, _turn(st["k"], cs, c["turned"], c["pairs"]))
    _plain_store(st["cache"][1], at, st["v"])
    return _turn(st["q"], cs, c["turned"], c["pairs"]).bfloat16(), _plain_load(st["cache"][0], at), _plain_load(st["cache"][1], at)


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


def _plain_product(st):
    c = st["c"]
    y = st["x"].float() @ _plain_weight(st["chunks"], c["kind"], c["rows"], c["cols"]).T
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if c["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = y * 0.5 * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = y * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if st["mul"] is not None:
        y = y * st["mul"].float()
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.bfloat16()


_run_own = dict(shared=_own_shared, cross=_own_cross, rotary=_own_rotary, product=_own_product)
_run_plain = dict(shared=_plain_attention, cross=_plain_attention, rotary=_plain_rotary, product=_plain_product)


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


def _exact_attention(c, seed):
    i = _cache_inputs(c, seed)
    q, scale, group = _query(c, i), 1 / math.sqrt(c["dim"]), c["heads"] // c["kv_heads"]
    outs, lses, begin, known = [], [], 0, {}
    for n, t, (pre, mine) in zip(i["n"], i["t"], i["parts"]):
        if id(pre) not in known:
            known = {id(pre): (_kept(pre[0]), _kept(pre[1]))}
        k, v = (torch.cat([known[id(pre)][w], _kept(mine[w])]) for w in (0, 1))
        qb = q[begin:begin + t].double()
        hidden = torch.zeros(t, n, dtype=torch.bool, device=DEV)
        if c["op"] == "shared":
            hidden = torch.arange(n, device=DEV)[None] > torch.arange(n - t, n, device=DEV)[:, None]
        o, l = torch.empty_like(qb), torch.empty(t, c["heads"], dtype=torch.float64, device=DEV)
        for h in range(c["heads"]):
            logits = (qb[:, h] @ k[:, h // group].T * scale).masked_fill(hidden, -math.inf)
            l[:, h] = torch.logsumexp(logits, 1)
            o[:, h] = torch.exp(logits - l[:, h:h + 1]) @ v[:, h // group]
        outs.append(o)
        lses.append(l)
        begin += t
    return torch.cat(outs), torch.cat(lses)


def _exact_rotary(c, seed):
    i = _rotary_inputs(c, seed)
    pos = torch.cat([torch.arange(n - t, n, device=DEV) for n, t in zip(i["n"], i["t"])])
    half = c["turned"] // 2
    one = [2 * j if c["pairs"] else j for j in range(half)]
    two = [2 * j + 1 if c["pairs"] else j + half for j in range(half)]
    cos, sin = i["turns"][pos, None, :, 0].double(), i["turns"][pos, None, :, 1].double()
    qx, kx = i["q"].double(), i["k"].float()
    q = qx.clone()
    q[..., one] = qx[..., one] * cos - qx[..., two] * sin
    q[..., two] = qx[..., one] * sin + qx[..., two] * cos
    # the keys that are quantised are numbers of 32 bits: products and sums rounded one by one
    k, each = kx.clone(), lambda x, y: (x.double() * y).float().double()  # noqa: E731
    k[..., one] = (each(kx[..., one], cos) - each(kx[..., two], sin)).float()
    k[..., two] = (each(kx[..., two], cos) + each(kx[..., one], sin)).float()
    return q, _kept(k), _kept(i["v"])


def exact(c, seed):
    if c["op"] in ("shared", "cross"):
        return _exact_attention(c, seed)
    if c["op"] == "rotary":
        return _exact_rotary(c, seed)
    i = _product_inputs(c, seed)
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
    if c["bias"]:
        y += i["bias"].double()
    y = dict(none=lambda z: z, relu=lambda z: z.clamp(min=0), silu=lambda z: z * torch.sigmoid(z),
             gelu=lambda z: z * torch.special.ndtr(z),
             gelu_tanh=lambda z: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))[c["act"]](y)
    if c["mul"]:
        y *= i["mul"].double()
    return y + i["residual"].double() if c["residual"] else y
