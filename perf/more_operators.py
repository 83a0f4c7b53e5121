"""Cases that time rotary positions, the 16-bit paged K/V cache and attention of new tokens
over it: the calls that surround the prefill over pages.

A rotation turns pair j of a row by the angle position * inv_freq[j], with the position of the
pair's axis (one axis for text; time, height and width for images and video).  Pairs are the
two halves of the rotated part, or neighbours where they are interleaved; elements behind the
last pair pass.  Cached rows are 16-bit and live in pages that a block table names.

Each case runs in a plain form of elementary torch operations (``own`` false) or through the
package's ``rotary``, ``cache16_write`` and ``decode16`` (``own`` true), on the same inputs.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, tokens=1, longest=1, ragged=False, heads_kv=8, group=4, d=128,
             page=64, dtype="bf16", pages="phtd", packed=False, q_len=1, pairs=64, axes=1,
             interleaved=False, inverse=False, rotate=True, queries=True)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # The queries and keys of a long prompt, at the heads of the repository's flagship layer.
        _case("rotary", "rotary_prompt_32k", tokens=32768, longest=32768),
        # Clips of uneven lengths packed together, each token with a time, a row and a column;
        # half precision, small heads, as many KV heads as query heads.
        _case("rotary", "rotary_video_fp16", batch=6, tokens=1777, longest=40000, ragged=True,
              packed=True, heads_kv=16, group=1, d=64, pairs=32, axes=3, dtype="fp16"),
        # The gradient of a rotation of half of each row, neighbours paired.
        _case("rotary", "rotary_gradient", batch=3, tokens=5003, longest=5003, pairs=32,
              interleaved=True, inverse=True),
        # One decode step of one conversation: latency only.
        _case("write", "append_one", longest=4097),
        # One decode step of a full batch: a token each, at 256 different positions.
        _case("write", "append_256", batch=256, longest=4096, ragged=True),
        # A long prompt on its way to the prefill over pages: queries and keys rotated, keys and
        # values into their pages, at the length of the repository's flagship layer.
        _case("write", "write_prompt_128k", tokens=131072, longest=131072, page=128),
        # Chunks of uneven prompts packed together behind what their sequences hold already,
        # pages laid out token first that end inside every tile, image positions.
        _case("write", "write_packed_fp16", batch=9, tokens=1531, longest=2600, ragged=True,
              packed=True, heads_kv=5, d=64, pairs=24, axes=2, page=48, dtype="fp16",
              pages="pthd"),
        # One conversation with a short history: latency.
        _case("decode", "decode_1x4k", longest=4097),
        # One conversation with a very long history: the work has to be split over its length.
        _case("decode", "decode_1x128k", longest=131072, page=128),
        # A full serving batch of medium histories: the largest amount of cache read at once.
        _case("decode", "decode_64x16k", batch=64, longest=16384, ragged=True),
        # Many short sequences, small heads, eight query heads to a KV head.
        _case("decode", "decode_256x600", batch=256, longest=600, ragged=True, heads_kv=2,
              group=8, d=64, page=16, dtype="fp16"),
        # Five proposed tokens a sequence verified at once (a causal window at the end), pages
        # laid out as the prefill's default.
        _case("decode", "verify_16x32k", batch=16, longest=32766, ragged=True, q_len=5, page=32,
              pages="pthd"),
    ]


def draw(rng):
    op = rng.choice(["rotary", "write", "decode", "decode"])
    d = rng.choice([64, 128])
    heads_kv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    batch = int(2 ** rng.uniform(0, 8))
    q_len = rng.choice([1, 1, 1, 1, 2, 3, 4, 5, 8])
    # no more elements, and no more products, than the largest listed cases have
    longest = int(2 ** rng.uniform(0, 17.01))
    if op == "decode":
        longest = max(1, min(longest, min(2 ** 32 // (group * q_len), 2 ** 29)
                             // (batch * heads_kv * d)))
    else:
        longest = max(1, min(longest, 2 ** 29 // (batch * heads_kv * (group + 2) * d)))
    tokens = 1 if rng.random() < 0.3 else max(1, int(2 ** rng.uniform(0, math.log2(longest + 1))))
    return _case(op, batch=batch, longest=longest, tokens=min(tokens, longest),
                 ragged=rng.random() < 0.75, heads_kv=heads_kv, group=group, d=d,
                 page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=rng.choice(["bf16", "fp16"]),
                 pages=rng.choice(["phtd", "phtd", "pthd"]), packed=rng.random() < 0.5,
                 q_len=q_len, pairs=rng.choice([d // 2, d // 2, d // 2, 8, 16, d // 2 - 8]),
                 axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4,
                 inverse=rng.random() < 0.4, rotate=rng.random() < 0.8,
                 queries=rng.random() < 0.8)


def _lengths(c):
    """Tokens that each sequence has, and how many of them (its last ones) the call takes; both
    follow from the case alone."""
    r = random.Random("%s %s %s" % (c["batch"], c["longest"], c["heads_kv"]))
    n, most = c["batch"], c["longest"]
    lens = [most] * n
    if c["ragged"]:
        lens = [most] + [r.randint(max(1, most // 16), most) for _ in range(n - 1)]
    take = [min(c["tokens"], x) for x in lens]
    if c["packed"]:
        take = [min(x, r.randint(0, 2 * c["tokens"])) for x in lens]
        take[0] = max(1, take[0])
    elif c["op"] != "decode":
        lens = [max(x, c["tokens"]) for x in lens]  # a rectangle of `tokens` each
        take = [c["tokens"]] * n
    return lens, take


def work(c):
    lens, take = _lengths(c)
    heads = c["heads_kv"] * c["group"]
    row = 2 * c["d"]
    if c["op"] == "decode":
        seen = sum(max(0, x - c["q_len"] + 1 + i) for x in lens for i in range(c["q_len"]))
        tables = 4 * sum(-(-x // c["page"]) for x in lens)
        return {"bytes": 2 * sum(lens) * c["heads_kv"] * row +
                2 * c["batch"] * c["q_len"] * heads * row + tables,
                "flops": 4 * seen * heads * c["d"]}
    n = sum(take)
    if c["op"] == "rotary":
        turned, rows = n * (heads + c["heads_kv"]), n * (heads + c["heads_kv"])
    else:
        rotated_q = heads if c["rotate"] and c["queries"] else 0
        turned = n * (rotated_q + c["heads_kv"]) if c["rotate"] else 0
        rows = n * (rotated_q + 2 * c["heads_kv"])
    return {"bytes": 2 * rows * row + 4 * n * c["axes"], "flops": 6 * turned * c["pairs"]}


# ------------------------------------------------------------------------------------ inputs
def _axes(c):
    """The axis of each pair: runs of uneven lengths, as for time, height and width."""
    if c["axes"] == 1:
        return None
    first = c["pairs"] // 4 if c["axes"] == 3 else c["pairs"] // 2
    rest = c["pairs"] - first
    second = (rest + 1) // 2 if c["axes"] == 3 else rest
    return (0,) * first + (1,) * second + (2,) * (rest - second)


def _rows(g, shape, heads_at, kind):
    """Queries, keys or values as a model's projections leave them: keys with a few strong
    channels, values flat."""
    x = torch.randn(shape, generator=g, device="cuda")
    if kind == "v":
        x *= 0.7
    elif kind == "k":
        one = [n if i in (heads_at, len(shape) - 1) else 1 for i, n in enumerate(shape)]
        strong = torch.randn(one, generator=g, device="cuda").abs()
        x *= 0.5 + 0.5 * strong + 3.0 * (strong > 2.3)
    return x


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    lens, take = _lengths(c)
    B, H, d, page, T = c["batch"], c["heads_kv"], c["d"], c["page"], TYPES[c["dtype"]]
    s = {"case": c, "T": T}
    s["seqlens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c["op"] != "rotary":
        per = [-(-x // page) for x in lens]
        pool = sum(per) + 3
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(B, max(per) + 1, dtype=torch.int32, device="cuda")
        at = torch.tensor([0] + per).cumsum(0)[:-1].to("cuda")
        col = torch.arange(max(per), device="cuda")
        used = col[None] < torch.tensor(per, device="cuda")[:, None]
        table[:, :-1] = torch.where(used, order[(at[:, None] + col[None]).clamp(max=pool - 1)], 0)
        s["table"] = table
        inner = (H, page) if c["pages"] == "phtd" else (page, H)
        for n in ("k", "v"):
            if c["op"] == "write":  # the pool as an allocator leaves it
                s[n + "_pool"] = torch.zeros(pool, *inner, d, dtype=T, device="cuda")
            else:
                s[n + "_pool"] = _rows(g, (pool, *inner, d), 1 if c["pages"] == "phtd" else 2,
                                       n).to(T)
    if c["op"] == "decode":
        s["q"] = _rows(g, (B, H * c["group"], c["q_len"], d), 1, "q").to(T)
        return s
    s["start"] = s["seqlens"] - torch.tensor(take, dtype=torch.int32, device="cuda")
    s["cu"] = None
    s["total"] = n = sum(take)
    if c["packed"]:
        s["cu"] = torch.tensor([0] + take).cumsum(0).to("cuda", torch.int32)
    # packed: [tokens, heads, d]; else [batch, heads, tokens, d] as the prefill takes them
    for name, heads in (("q", H * c["group"]), ("k", H), ("v", H)):
        shape = (n, heads, d) if c["packed"] else (B, heads, c["tokens"], d)
        s[name] = _rows(g, shape, 1, name).to(T)
    s["inv_freq"] = 10000.0 ** (-torch.arange(c["pairs"], device="cuda") / c["pairs"])
    s["axes"] = _axes(c)
    s["positions"] = None
    if c["axes"] > 1:
        # a clip's grid: the place in time advances once a frame, rows and columns within it
        where = (n,) if c["packed"] else (B, c["tokens"])
        t = torch.arange(n, device="cuda").view(where)
        wide = torch.randint(5, 40, (), generator=g, device="cuda")
        tall = torch.randint(3, 30, (), generator=g, device="cuda")
        far = torch.randint(0, c["longest"] + 1, (), generator=g, device="cuda")
        grid = [far + t // (wide * tall), far + t // wide % tall, far + t % wide]
        if c["axes"] == 2:
            grid = grid[1:]
        s["positions"] = torch.stack(grid).to(torch.int32).contiguous()
    return s


# -------------------------------------------------------------------------------- plain form
def _owner(s):
    """(sequence, position) of every token that the call takes, in order."""
    c = s["case"]
    if s["cu"] is None:
        b = torch.arange(c["batch"], device="cuda").repeat_interleave(c["tokens"])
        i = torch.arange(c["tokens"], device="cuda").repeat(c["batch"])
    else:
        t = torch.arange(s["total"], device="cuda")
        b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
        i = t - s["cu"].long()[b]
    return b, s["start"].long()[b] + i


def _plain_angles(s):
    """cos and sin [tokens, pairs] in fp32, from angles in 64 bits."""
    c = s["case"]
    if s["positions"] is None:
        pos = _owner(s)[1][:, None].expand(-1, c["pairs"])
    else:
        axis = torch.tensor(s["axes"], device="cuda")
        pos = s["positions"].flatten(1)[axis].T
    angle = pos.double() * s["inv_freq"].double()
    if c["inverse"] and c["op"] == "rotary":
        angle = -angle
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_turn(s, x, cos, sin):
    c = s["case"]
    P = c["pairs"]
    if s["cu"] is None:  # [batch, heads, tokens, d]
        cos, sin = (a.view(c["batch"], 1, c["tokens"], P) for a in (cos, sin))
    else:  # [tokens, heads, d]
        cos, sin = cos[:, None], sin[:, None]
    y = x.float()
    out = y.clone()
    if c["interleaved"]:
        a, b = y[..., 0:2 * P:2], y[..., 1:2 * P:2]
        out[..., 0:2 * P:2] = a * cos - b * sin
        out[..., 1:2 * P:2] = b * cos + a * sin
    else:
        a, b = y[..., :P], y[..., P:2 * P]
        out[..., :P] = a * cos - b * sin
        out[..., P:2 * P] = b * cos + a * sin
    return out.to(s["T"])


def _plain_rotary(s):
    cos, sin = _plain_angles(s)
    return _plain_turn(s, s["q"], cos, sin), _plain_turn(s, s["k"], cos, sin)


def _plain_write(s):
    c = s["case"]
    q, k, v = None, s["k"], s["v"]
    if c["rotate"]:
        cos, sin = _plain_angles(s)
        k = _plain_turn(s, k, cos, sin)
        if c["queries"]:
            q = _plain_turn(s, s["q"], cos, sin)
    b, pos = _owner(s)
    page, row = s["table"].long()[b, pos // c["page"]], pos % c["page"]
    for pool, x in ((s["k_pool"], k), (s["v_pool"], v)):
        if s["cu"] is None:  # -> [tokens, heads, d]
            x = x.transpose(1, 2).flatten(0, 1)
        (pool.transpose(1, 2) if c["pages"] == "phtd" else pool)[page, row] = x
    pools = (s["k_pool"], s["v_pool"])
    return pools if q is None else (q,) + pools


def _plain_decode(s):
    c = s["case"]
    H, d, n = c["heads_kv"], c["d"], c["q_len"]
    pages = s["table"][:, :-1].long()
    kv = []
    for name in ("k", "v"):
        x = s[name + "_pool"][pages].float()
        if c["pages"] == "pthd":
            x = x.transpose(2, 3)
        kv.append(x.transpose(1, 2).flatten(2, 3))  # [batch, heads, keys, d]
    k, v = kv
    q = s["q"].float().unflatten(1, (H, c["group"])).flatten(2, 3)
    scores = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    scores = scores.unflatten(2, (c["group"], n))
    key = torch.arange(k.shape[2], device="cuda")
    last = s["seqlens"].long()[:, None] - n + torch.arange(n, device="cuda")
    hidden = (key[None, None] > last[..., None])[:, None, None]
    scores = scores.masked_fill(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v) / total.clamp(min=1e-30).flatten(2, 3)
    out = out.unflatten(2, (c["group"], n)).flatten(1, 2).to(s["T"])
    lse = (top + torch.log(total)).squeeze(-1).flatten(1, 2)  # [batch, query heads, q_len]
    return out, lse.transpose(0, 1).flatten(1)


# ------------------------------------------------------------------------------ the package's
def _own(s):
    import block_sparse_gated_gb300 as bsfa
    c = s["case"]
    if c["op"] == "decode":
        cache = bsfa.KVCache16(s["k_pool"], s["v_pool"], c["pages"])
        r = bsfa.decode16(s["q"], cache, s["table"], s["seqlens"], max_seqlen=c["longest"],
                          return_lse=True)
        return r["out"], r["lse"]
    where = {"start": s["start"], "positions": s["positions"]}
    if s["cu"] is not None:
        where.update(cu_seqlens=s["cu"], layout="thd")
    rope = bsfa.Rope(s["inv_freq"], s["axes"], c["interleaved"])
    if c["op"] == "rotary":
        return bsfa.rotary(rope, s["q"], s["k"], inverse=c["inverse"], **where)
    cache = bsfa.KVCache16(s["k_pool"], s["v_pool"], c["pages"])
    if not c["rotate"]:
        rope, where["positions"] = None, None
    q = bsfa.cache16_write(cache, s["k"], s["v"], s["table"], rope=rope,
                           q=s["q"] if c["rotate"] and c["queries"] else None, **where)
    pools = (s["k_pool"], s["v_pool"])
    return pools if q is None else (q,) + pools


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_rotary(s) if op == "rotary" else _plain_write(s) if op == "write" else \
        _plain_decode(s)


# -------------------------------------------------------------------------------- in 64 bits
def _exact_rotated(s, x, sign):
    """fp64 rows as complex numbers, each times a number of size one."""
    c = s["case"]
    lens, take = _lengths(c)
    P = c["pairs"]
    if s["positions"] is None:
        turns = torch.cat([torch.arange(n - m, n, dtype=torch.float64) for n, m in
                           zip(lens, take)]).to("cuda")
        turns = turns[:, None] * s["inv_freq"].double()[None]
    else:
        place = s["positions"].reshape(c["axes"], -1).double()
        turns = torch.empty(place.shape[1], P, dtype=torch.float64, device="cuda")
        for j in range(P):
            turns[:, j] = place[s["axes"][j]] * s["inv_freq"][j].double()
    unit = torch.polar(torch.ones_like(turns), sign * turns)
    if c["packed"]:
        unit = unit[:, None, :]
    else:
        unit = unit.reshape(c["batch"], c["tokens"], P)[:, None]
    out = x.double()
    if c["interleaved"]:
        z = torch.view_as_complex(out[..., :2 * P].unflatten(-1, (P, 2)).contiguous()) * unit
        turned = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(out[..., :P], out[..., P:2 * P]) * unit
        turned = torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, out[..., 2 * P:]], -1)


def _exact_write(c, s):
    lens, take = _lengths(c)
    k = _exact_rotated(s, s["k"], 1.0) if c["rotate"] else s["k"].double()
    out = [_exact_rotated(s, s["q"], 1.0)] if c["rotate"] and c["queries"] else []
    table = s["table"].tolist()
    page, spots = c["page"], []
    for b in range(c["batch"]):
        for t in range(lens[b] - take[b], lens[b]):
            spots.append(table[b][t // page] * page + t % page)
    spots = torch.tensor(spots, device="cuda")
    for x, pool in ((k, s["k_pool"]), (s["v"].double(), s["v_pool"])):
        # one row of a flat pool for each (page, token), the heads beside each other
        token_first = pool.double() if c["pages"] == "pthd" else pool.double().transpose(1, 2)
        flat = token_first.reshape(-1, c["heads_kv"], c["d"])
        rows = x if c["packed"] else x.transpose(1, 2).reshape(-1, c["heads_kv"], c["d"])
        flat = flat.index_copy(0, spots, rows).reshape(token_first.shape)
        out.append((flat if c["pages"] == "pthd" else flat.transpose(1, 2)).contiguous())
    return tuple(out)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rotary":
        sign = -1.0 if c["inverse"] else 1.0
        return _exact_rotated(s, s["q"], sign), _exact_rotated(s, s["k"], sign)
    if c["op"] == "write":
        return _exact_write(c, s)
    lens, _ = _lengths(c)
    n, outs, logs = c["q_len"], [], []
    for b in range(c["batch"]):
        pages = s["table"][b, :-(-lens[b] // c["page"])].long()
        k, v = (s[x + "_pool"][pages] for x in ("k", "v"))
        if c["pages"] == "phtd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        k, v = (x.reshape(-1, c["heads_kv"], c["d"])[:lens[b]].double() for x in (k, v))
        q = s["q"][b].double().reshape(c["heads_kv"], -1, c["d"])
        w = torch.einsum("hrd,khd->hrk", q, k) / math.sqrt(c["d"])
        w = w.reshape(c["heads_kv"] * c["group"], n, -1)
        for i in range(n):
            w[:, i, max(0, lens[b] - n + 1 + i):] = -math.inf
        logs.append(torch.logsumexp(w, -1))
        w = torch.nan_to_num(torch.softmax(w, -1), nan=0.0).reshape(c["heads_kv"], -1, lens[b])
        outs.append(torch.einsum("hrk,khd->hrd", w, v).reshape(-1, n, c["d"]))
    return torch.stack(outs), torch.cat(logs, -1)
