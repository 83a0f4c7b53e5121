"""Cases that time the 4-bit K/V cache: writing keys and values into its pages, reading them
back, and attention of new tokens over it.

A cached row (one token of one KV head) of head dimension d is d e2m1 codes, two to a byte with
the even element in the low half, and one e4m3 scale for every 16 elements; a value is
code * scale * 2**exponent, with one exponent for each KV head (0 where there is none).  Rows
live in pages that a block table names.

Each case runs in a plain form of elementary torch operations (``own`` false) or through the
package's ``cache4_write``, ``cache4_read`` and ``decode4`` (``own`` true), on the same inputs.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 16  # elements that share a scale


# ------------------------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, tokens=1, longest=1, ragged=False, heads_kv=8, group=4, d=128,
             page=64, dtype="bf16", pages="phtd", packed=False, exponents=False, q_len=1)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # One decode step of one conversation: its new token enters the cache and comes back as
        # the value that later steps will see.  Latency only.
        _case("write", "append_one", longest=4097),
        # One decode step of a full batch: a token each, at 256 different positions.
        _case("write", "append_256", batch=256, longest=4096, ragged=True),
        # A long prompt after its prefill, at the length of the repository's flagship layer.
        _case("write", "write_prompt_128k", tokens=131072, longest=131072, page=128),
        # Prompts of uneven lengths packed together, half precision, small heads, values far
        # below one (per-head exponents), pages that end inside every tile.
        _case("write", "write_packed_fp16", batch=9, tokens=1531, longest=2600, ragged=True,
              packed=True, heads_kv=5, d=64, page=48, dtype="fp16", exponents=True),
        # The cache of a long prompt back in 16 bits, for a prefill over all of it.
        _case("read", "read_prompt_128k", tokens=131072, longest=131072, page=128),
        # Uneven sequences read back packed from pages laid out token first.
        _case("read", "read_packed_fp16", batch=9, tokens=1531, longest=2600, ragged=True,
              packed=True, heads_kv=5, d=64, page=48, dtype="fp16", pages="pthd",
              exponents=True),
        # One conversation with a short history: latency.
        _case("decode", "decode_1x4k", longest=4097),
        # One conversation with a very long history: the work has to be split over its length.
        _case("decode", "decode_1x128k", longest=131072, page=128),
        # Eight sequences between 4K and 64K, the lengths of the repository's packed workload.
        _case("decode", "decode_8x64k", batch=8, longest=65536, ragged=True, page=128),
        # A full serving batch of medium histories: the largest amount of cache read at once.
        _case("decode", "decode_64x16k", batch=64, longest=16384, ragged=True),
        # Many short sequences, small heads, eight query heads to a KV head.
        _case("decode", "decode_256x600", batch=256, longest=600, ragged=True, heads_kv=2,
              group=8, d=64, page=16, dtype="fp16"),
        # Five proposed tokens a sequence verified at once (a causal window at the end).
        _case("decode", "verify_16x32k", batch=16, longest=32766, ragged=True, q_len=5, page=32,
              exponents=True),
    ]


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode"])
    d = rng.choice([64, 128])
    heads_kv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    batch = int(2 ** rng.uniform(0, 8))
    q_len = rng.choice([1, 1, 1, 1, 2, 3, 4, 5, 8])
    # no more elements, and no more products, than the largest listed cases have
    most = 2 ** 32 // (group * q_len) if op == "decode" else 2 ** 27
    longest = int(2 ** rng.uniform(0, 17.01))
    longest = max(1, min(longest, min(most, 2 ** 29) // (batch * heads_kv * d)))
    tokens = 1 if rng.random() < 0.4 else max(1, int(2 ** rng.uniform(0, math.log2(longest + 1))))
    return _case(op, batch=batch, longest=longest, tokens=min(tokens, longest),
                 ragged=rng.random() < 0.75, heads_kv=heads_kv, group=group, d=d,
                 page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=rng.choice(["bf16", "fp16"]),
                 pages=rng.choice(["phtd", "phtd", "pthd"]), packed=rng.random() < 0.5,
                 exponents=rng.random() < 0.4, q_len=q_len)


def _lengths(c):
    """Tokens that each sequence has in the cache, and how many of them (its last ones) a
    write or a read takes; both follow from the case alone."""
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
    row = c["d"] // 2 + c["d"] // GROUP
    if c["op"] == "decode":
        heads = c["heads_kv"] * c["group"]
        queries = c["batch"] * c["q_len"] * heads * c["d"]
        seen = sum(max(0, x - c["q_len"] + 1 + i) for x in lens for i in range(c["q_len"]))
        tables = 4 * sum(-(-x // c["page"]) for x in lens)
        return {"bytes": 2 * sum(lens) * c["heads_kv"] * row + 2 * 2 * queries + tables,
                "flops": 4 * seen * heads * c["d"]}
    rows = 2 * sum(take) * c["heads_kv"]
    wide = rows * 2 * c["d"]
    if c["op"] == "write":  # 16 bits in, codes and scales out, the values they stand for out
        return {"bytes": 2 * wide + rows * row, "flops": 4 * rows * c["d"]}
    return {"bytes": wide + rows * row, "flops": 2 * rows * c["d"]}


# ------------------------------------------------------------------------------------ inputs
def _rows(g, shape, exponents, heads_at, value):
    """Keys or values as a model's projections leave them: keys with a few strong channels,
    values flat; small in scale where the heads carry exponents."""
    x = torch.randn(shape, generator=g, device="cuda")
    if value:
        x *= 0.7
    else:
        one = [n if i in (heads_at, len(shape) - 1) else 1 for i, n in enumerate(shape)]
        strong = torch.randn(one, generator=g, device="cuda").abs()
        x *= 0.5 + 0.5 * strong + 3.0 * (strong > 2.3)
    return x * 2.0 ** -9 if exponents else x


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    lens, take = _lengths(c)
    B, H, d, page, T = c["batch"], c["heads_kv"], c["d"], c["page"], TYPES[c["dtype"]]
    per = [-(-x // page) for x in lens]
    pool = sum(per) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B, max(per) + 1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0] + per).cumsum(0)[:-1].to("cuda")
    col = torch.arange(max(per), device="cuda")
    used = col[None] < torch.tensor(per, device="cuda")[:, None]
    table[:, :-1] = torch.where(used, order[(at[:, None] + col[None]).clamp(max=pool - 1)], 0)
    s = {"case": c, "table": table, "T": T,
         "seqlens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "k_exp": None, "v_exp": None}
    if c["exponents"]:
        s["k_exp"] = torch.randint(-10, -7, (H,), generator=g, device="cuda", dtype=torch.int32)
        s["v_exp"] = torch.randint(-11, -8, (H,), generator=g, device="cuda", dtype=torch.int32)
    inner = (H, page) if c["pages"] == "phtd" else (page, H)
    if c["op"] == "write":
        # the pool as an allocator leaves it
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros(pool, *inner, d // 2, dtype=torch.uint8, device="cuda")
            s[n + "_scale"] = torch.zeros(pool, *inner, d // GROUP, dtype=torch.float8_e4m3fn,
                                          device="cuda")
    else:
        for n in ("k", "v"):
            x = _rows(g, (pool, *inner, d), c["exponents"], 1 if c["pages"] == "phtd" else 2,
                      n == "v")
            s[n + "_codes"], s[n + "_scale"] = _quantise(x, s[n + "_exp"], c["pages"])
            del x
    s["start"] = s["seqlens"] - torch.tensor(take, dtype=torch.int32, device="cuda")
    s["cu"] = None
    s["total"] = sum(take)
    if c["packed"]:
        s["cu"] = torch.tensor([0] + take).cumsum(0).to("cuda", torch.int32)
    if c["op"] == "write":
        # packed: [tokens, heads, d]; else [batch, heads, tokens, d] as the prefill takes them
        shape = (sum(take), H, d) if c["packed"] else (B, H, c["tokens"], d)
        for n in ("k", "v"):
            s[n] = _rows(g, shape, c["exponents"], 1, n == "v").to(T)
    if c["op"] == "decode":
        q = torch.randn(B, H * c["group"], c["q_len"], d, generator=g, device="cuda")
        s["q"] = (q * (2.0 ** 9 if c["exponents"] else 1.0)).to(T)
    return s


# -------------------------------------------------------------------------------- plain form
def _head_factor(exp, layout, sign):
    if exp is None:
        return 1.0
    f = torch.exp2(sign * exp.float())
    return f[:, None, None] if layout == "phtd" else f[:, None]


def _quantise(x, exp, layout):
    """fp32 [.., heads, rows, d] ("phtd") or [.., rows, heads, d] -> codes, scales."""
    x = x.float() * _head_factor(exp, layout, -1.0)
    x = x.unflatten(-1, (-1, GROUP))
    scale = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    scale = scale.clamp(min=2.0 ** -9)
    y = x.abs() / scale[..., None]
    code = (y > 0.25).to(torch.uint8)
    code += y >= 0.75  # halfway between two codes: the even one
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5.0
    code += torch.signbit(x).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(torch.float8_e4m3fn)


def _values(codes, scale, exp, layout):
    """The fp32 values of codes and scales laid out as in the pool."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    size = (code & 7).float()
    big = torch.exp2((size / 2).floor() - 1.0) * (1.0 + 0.5 * (size % 2))
    x = torch.where(size < 2, 0.5 * size, big)
    x = torch.where(code >= 8, -x, x)
    x = x.unflatten(-1, (-1, GROUP)) * scale.float()[..., None]
    return x.flatten(-2) * _head_factor(exp, layout, 1.0)


def _slots(s):
    """(sequence, page, row in it) of every token that a write or a read takes."""
    c = s["case"]
    if s["cu"] is None:
        b = torch.arange(c["batch"], device="cuda").repeat_interleave(c["tokens"])
        i = torch.arange(c["tokens"], device="cuda").repeat(c["batch"])
    else:
        t = torch.arange(s["total"], device="cuda")
        b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
        i = t - s["cu"].long()[b]
    pos = s["start"].long()[b] + i
    return s["table"].long()[b, pos // c["page"]], pos % c["page"]


def _plain_write(s):
    c = s["case"]
    page, row = _slots(s)
    out = []
    for n in ("k", "v"):
        x = s[n]
        if s["cu"] is None:  # -> [tokens, heads, d]
            x = x.transpose(1, 2).flatten(0, 1)
        codes, scale = _quantise(x, s[n + "_exp"], "pthd")
        held, held_scale = s[n + "_codes"], s[n + "_scale"].view(torch.uint8)
        if c["pages"] == "phtd":
            held, held_scale = held.transpose(1, 2), held_scale.transpose(1, 2)
        held[page, row] = codes
        held_scale[page, row] = scale.view(torch.uint8)
        out.append(_values(codes, scale, s[n + "_exp"], "pthd").to(s["T"]))
    return _wide(s, out)


def _plain_read(s):
    page, row = _slots(s)
    out = []
    for n in ("k", "v"):
        codes, scale = s[n + "_codes"], s[n + "_scale"].view(torch.uint8)
        if s["case"]["pages"] == "phtd":
            codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
        scale = scale[page, row].view(torch.float8_e4m3fn)
        out.append(_values(codes[page, row], scale, s[n + "_exp"], "pthd").to(s["T"]))
    return _wide(s, out)


def _wide(s, rows):
    """[tokens, heads, d] as the call lays it out."""
    if s["cu"] is not None:
        return tuple(rows)
    c = s["case"]
    return tuple(x.unflatten(0, (c["batch"], c["tokens"])).transpose(1, 2).contiguous()
                 for x in rows)


def _plain_decode(s):
    c = s["case"]
    H, d, n = c["heads_kv"], c["d"], c["q_len"]
    pages = s["table"][:, :-1].long()
    kv = []
    for name in ("k", "v"):
        x = _values(s[name + "_codes"][pages], s[name + "_scale"].view(torch.uint8)[pages].view(
            torch.float8_e4m3fn), s[name + "_exp"], c["pages"])
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
    return out.unflatten(2, (c["group"], n)).flatten(1, 2).to(s["T"])


# ------------------------------------------------------------------------------ the package's
def _own(s):
    import block_sparse_gated_gb300 as bsfa
    c = s["case"]
    cache = bsfa.KVCache4(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_exp"],
                          s["v_exp"], c["pages"])
    if c["op"] == "decode":
        return bsfa.decode4(s["q"], cache, s["table"], s["seqlens"],
                            max_seqlen=c["longest"])["out"]
    where = {"start": s["start"]}
    if s["cu"] is not None:
        where.update(cu_seqlens=s["cu"], layout="thd")
    if c["op"] == "write":
        bsfa.cache4_write(cache, s["k"], s["v"], s["table"], **where)
    size = {"seqlen": c["tokens"]} if s["cu"] is None else {"total": s["total"]}
    return bsfa.cache4_read(cache, s["table"], dtype=s["T"], **where, **size)


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_write(s) if op == "write" else _plain_read(s) if op == "read" else \
        _plain_decode(s)


# -------------------------------------------------------------------------------- in 64 bits
_SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _near(a, least, digits, most):
    """Nonnegative fp64 `a` rounded to `digits` bits after the leading one, half to even, with
    2**least the smallest normal number and `most` the largest value."""
    e = torch.frexp(a).exponent.to(torch.float64) - 1
    unit = torch.exp2(e.clamp(min=least) - digits)
    return (torch.round(a / unit) * unit).clamp(max=most)


def _exact_stored(x, exp):
    """fp64 values [tokens, heads, d] that stand in the cache for x."""
    f = torch.ones(x.shape[1], dtype=torch.float64, device="cuda")
    if exp is not None:
        f = torch.exp2(exp.double())
    f = f[:, None, None]
    y = x.double().reshape(*x.shape[:2], -1, GROUP) / f
    scale = _near(y.abs().amax(-1, keepdim=True) / 6, -6, 3, 448.0).clamp(min=2.0 ** -9)
    y = _near(y.abs() / scale, 0, 1, 6.0) * torch.sign(y)
    return (y * scale * f).reshape(x.shape)


def _exact_row(s, n, pages, count):
    """fp64 [heads, count, d] of one sequence's first tokens."""
    c = s["case"]
    sizes = torch.tensor(_SIZES + tuple(-x for x in _SIZES), dtype=torch.float64, device="cuda")
    byte = s[n + "_codes"][pages]
    x = torch.empty(*byte.shape[:-1], c["d"], dtype=torch.float64, device="cuda")
    x[..., 0::2] = sizes[(byte % 16).int()]
    x[..., 1::2] = sizes[(byte // 16).int()]
    scale = s[n + "_scale"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
    x *= scale.repeat_interleave(GROUP, -1)
    if c["pages"] == "phtd":
        x = x.transpose(0, 1)  # heads first
    else:
        x = x.permute(2, 0, 1, 3)
    x = x.reshape(c["heads_kv"], -1, c["d"])[:, :count]
    return x if s[n + "_exp"] is None else x * torch.exp2(s[n + "_exp"].double())[:, None, None]


def exact(c, seed):
    s = prepare(c, seed)
    lens, take = _lengths(c)
    out = {"k": [], "v": []}
    if c["op"] == "write":
        for n in out:
            x = s[n] if c["packed"] else s[n].transpose(1, 2).flatten(0, 1)
            y = _exact_stored(x, s[n + "_exp"])
            if not c["packed"]:
                y = y.reshape(c["batch"], c["tokens"], *x.shape[1:]).transpose(1, 2)
            out[n] = y.contiguous()
        return out["k"], out["v"]
    tables = s["table"].long()
    if c["op"] == "read":
        for n in out:
            for b in range(c["batch"]):
                x = _exact_row(s, n, tables[b, :-(-lens[b] // c["page"])], lens[b])
                x = x[:, lens[b] - take[b]:]
                out[n].append(x.transpose(0, 1) if c["packed"] else x)
        join = torch.cat if c["packed"] else torch.stack
        return join(out["k"]).contiguous(), join(out["v"]).contiguous()
    rows = []
    for b in range(c["batch"]):
        pages = tables[b, :-(-lens[b] // c["page"])]
        k, v = (_exact_row(s, n, pages, lens[b]) for n in ("k", "v"))
        q = s["q"][b].double().reshape(c["heads_kv"], -1, c["d"])
        w = torch.einsum("hrd,hkd->hrk", q, k) / math.sqrt(c["d"])
        w = w.reshape(c["heads_kv"] * c["group"], c["q_len"], -1)
        for i in range(c["q_len"]):
            w[:, i, max(0, lens[b] - c["q_len"] + 1 + i):] = -math.inf
        w = torch.nan_to_num(torch.softmax(w, -1), nan=0.0)
        w = w.reshape(c["heads_kv"], -1, lens[b])
        rows.append(torch.einsum("hrk,hkd->hrd", w, v).reshape(-1, c["q_len"], c["d"]))
    return torch.stack(rows)
