"""Workloads of the paged cache's operators: appending prepared keys and
values to a cache of pages (16-bit, or 4-bit e2m1 with a scale per 16
channels), attention over such a cache for single tokens, drafts and chunks of
prompt, and reading rows of a cache back.

``run`` computes an operator in its plain form (elementary torch operations in
binary32, rounded once at the end) or, with ``own`` set, through this
package's entry points; ``exact`` computes it in binary64 from its definition.
"""
import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}

# What a drawn case may cost: (query, key) pairs of all heads, values of a
# dense copy of the keys, rows of an append.
_MOST_PAIRS = 4 * 40 * 1024 * 16384
_MOST_KEYS = 32 * 8 * 32768 * 128
_MOST_APPEND = 32640 * 56 * 128


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _case(name, op, dtype, cache, batch, heads, kv_heads, dim, page, keys, **more):
    """keys: the most keys a sequence has; rows: query (or new) rows of the longest sequence."""
    c = {"name": name, "op": op, "dtype": dtype, "cache": cache, "batch": batch, "heads": heads, "kv_heads": kv_heads,
         "dim": dim, "page": page, "keys": keys, "rows": 1, "ragged": False, "idle": False, "rotary": 0, "axes": 1,
         "softcap": 0.0, "slopes": False, "prefix": False, "lens_seed": 0}
    c.update(more)
    return c


def listed():
    return [
        # One new token of one request joins a 4-bit cache: latency of the step before its attention.
        _case("append_token", "append", "fp16", "e2m1", 1, 16, 4, 64, 64, 4896, rotary=48, axes=3),
        # Prompts of five packed clips of uneven lengths, positions on a (t, h, w) grid, into 16-bit pages.
        _case("append_clips", "append", "bf16", "same", 5, 40, 8, 128, 64, 4080, rows=4080, ragged=True, rotary=96,
              axes=3, lens_seed=1),
        # A latent grid of 16x34x60 tokens into 4-bit pages.
        _case("append_latent_4bit", "append", "bf16", "e2m1", 1, 40, 8, 128, 128, 32640, rows=32640, rotary=96, axes=3),
        # One new token over one decoder tile's 4-bit cache: latency.
        _case("token_4bit", "attention", "fp16", "e2m1", 1, 16, 4, 64, 64, 4896),
        # One new token for each of 32 requests over 4-bit caches of uneven lengths, one slot idle.
        _case("token_batch_4bit", "attention", "bf16", "e2m1", 32, 40, 8, 128, 64, 32768, ragged=True, idle=True,
              lens_seed=2),
        # The same over 16-bit caches of small pages.
        _case("token_batch_16bit", "attention", "bf16", "same", 16, 40, 8, 128, 16, 32768, ragged=True, lens_seed=3),
        # One new token over one very long 4-bit cache: the keys have to be spread over the GPU.
        _case("token_long_4bit", "attention", "bf16", "e2m1", 1, 40, 8, 128, 128, 524288),
        # Four drafted tokens for each of 24 requests, capped scores.
        _case("drafts_4bit", "attention", "bf16", "e2m1", 24, 40, 8, 128, 64, 8192, rows=4, ragged=True, softcap=30.0,
              lens_seed=4),
        # Chunks of four prompts behind what their 4-bit caches hold already.
        _case("chunk_4bit", "attention", "bf16", "e2m1", 4, 40, 8, 128, 64, 16384, rows=1024, ragged=True, lens_seed=5),
        # Chunks of two prompts over 16-bit caches, a bias that grows with distance.
        _case("chunk_16bit", "attention", "fp16", "same", 2, 16, 4, 64, 64, 9792, rows=2448, ragged=True, slopes=True,
              lens_seed=6),
        # A few rows of one sequence read back: latency.
        _case("read_rows", "read", "fp16", "e2m1", 1, 16, 4, 64, 64, 288),
        # Four whole caches read back into dense 16-bit keys and values.
        _case("read_caches", "read", "bf16", "e2m1", 4, 40, 8, 128, 64, 32768, ragged=True, lens_seed=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(("append", "append", "token", "token", "few", "chunk", "chunk", "read"))
    cache = rng.choice(("e2m1", "e2m1", "same"))
    dim = rng.choice((32, 64, 64, 96, 128, 128) if cache == "e2m1" else (40, 64, 72, 96, 128, 128))
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 2, 4, 5))
    page = rng.choice((16, 32, 64, 128, 256))
    dtype = rng.choice(("fp16", "bf16"))
    seed = rng.randrange(1 << 20)
    ragged = rng.random() < 0.7
    if kind == "append":
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, _MOST_APPEND // ((heads + 2 * kv) * dim * batch)))
        axes = rng.choice((1, 3))
        c = _case(None, "append", dtype, cache, batch, heads, kv, dim, page, rows + rng.choice((0, 0, 100, 1000)),
                  rows=rows, ragged=ragged, rotary=dim if axes == 1 else dim // 8 * 6 // 6 * 6, axes=axes, lens_seed=seed)
    elif kind == "read":
        batch = _log(rng, 1, 16)
        c = _case(None, "read", dtype, cache, batch, heads, kv, dim, page,
                  _log(rng, 1, min(65536, _MOST_KEYS // 8 // (batch * kv * dim))), ragged=ragged, lens_seed=seed)
    else:
        batch = _log(rng, 1, 48) if kind != "chunk" else rng.choice((1, 2, 3, 6))
        keys = _log(rng, 1, min(262144 if kind == "token" else 32768, _MOST_KEYS // (batch * kv * 128)))
        rows = 1
        if kind == "few":
            rows = rng.randint(1, 12)
        elif kind == "chunk":
            rows = _log(rng, 8, max(8, min(4096, _MOST_PAIRS // (batch * heads * keys))))
        c = _case(None, "attention", dtype, cache, batch, heads, kv, dim, page, max(keys, rows), rows=rows, ragged=ragged,
                  idle=kind != "chunk" and batch > 4, softcap=rng.choice((0.0, 0.0, 20.0, 50.0)),
                  slopes=rng.random() < 0.3, prefix=kind == "chunk" and rng.random() < 0.3, lens_seed=seed)
    del c["name"]
    return c


def _lengths(case):
    """(rows, keys, prefix) of every sequence: its query or new rows, which are the last of its keys."""
    r = random.Random(case["lens_seed"])
    got = []
    for i in range(case["batch"]):
        rows, keys = case["rows"], case["keys"]
        if case["ragged"] and rows > 1:
            rows = rows if i == 0 else r.randint(max(1, rows // 4), rows)
        if case["ragged"]:
            keys = keys if i == 0 else max(rows, int(keys * r.uniform(0.25, 1.0)))
            if case["op"] == "append":
                keys = max(rows, case["keys"] - r.randint(0, case["keys"] // 8))
        if case["idle"] and i == case["batch"] // 2:
            rows, keys = 0, 0
        got.append((rows, keys, r.randint(0, keys // 3) if case["prefix"] else 0))
    return got


def _row_bytes(case):
    """Bytes of one head row of a cache."""
    return case["dim"] * 9 // 16 if case["cache"] == "e2m1" else 2 * case["dim"]


def work(case):
    lens = _lengths(case)
    rows, keys = sum(x[0] for x in lens), sum(x[1] for x in lens)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    kv = 2 * hk * _row_bytes(case)
    if case["op"] == "append":
        new = rows * (h + 2 * hk) * d
        got = {"bytes": 2 * new + 2 * rows * h * d + rows * kv, "flops": 20 * rows * (h + hk) * d}
        if case["cache"] == "e2m1":  # the new rows are read back as the values that they stand for
            got["bytes"] += rows * kv + 4 * rows * hk * d
        return got
    if case["op"] == "read":
        return {"bytes": keys * kv + 4 * case["batch"] * case["keys"] * hk * d, "flops": 2 * keys * hk * d}
    pairs = 0
    for n, k, prefix in lens:
        start = k - n
        wide = max(0, min(n, prefix - start))  # rows that see the whole prefix and no more
        pairs += wide * min(k, prefix) + sum(range(start + wide + 1, k + 1))
    return {"bytes": 4 * rows * h * d + 4 * rows * h + keys * kv, "flops": 4 * d * h * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFFFFFF)


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _e2m1(y):
    """Values and scales of 16-channel groups: float32 [..., groups, 16] to (codes 0..15, e4m3 scales)."""
    top = y.abs().amax(-1, keepdim=True)
    scale = (top * (1.0 / 6.0)).clamp(min=2.0 ** -9, max=448.0).to(torch.float8_e4m3fn)
    z = y * (1.0 / scale.float())
    a = z.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code + 8 * (z < 0), scale


def _value(codes, scales):
    """What packed codes [..., dim / 2] with scales [..., dim / 16] stand for, in binary32."""
    at = torch.tensor(_CODES + tuple(-c for c in _CODES), device="cuda")
    both = torch.stack([at[(codes & 15).long()], at[(codes >> 4).long()]], -1).flatten(-2)
    return (both.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _pages(case, n, g, normed):
    """n pages of one cache: [pages, kv_heads, page, dim] 16-bit, or (codes, scales).  Rows come from a bank, in any order."""
    hk, page, d, dt = case["kv_heads"], case["page"], case["dim"], _DT[case["dtype"]]
    bank = _randn((4096, d), g, torch.float32)
    if normed:
        bank *= 0.5 + torch.rand(d, generator=g, device="cuda")
    else:
        bank[:, torch.randint(0, d, (1,), generator=g, device="cuda")] *= 8.0
    at = torch.randint(0, 4096, (n, hk, page), generator=g, device="cuda")
    if case["cache"] != "e2m1":
        return bank.to(dt)[at], None
    code, scale = _e2m1(bank.to(dt).float().view(4096, d // 16, 16))
    code = code.view(4096, d).to(torch.uint8)
    code = code[:, 0::2] | (code[:, 1::2] << 4)
    return code[at], scale.view(torch.uint8).view(4096, d // 16)[at].view(torch.float8_e4m3fn)


def _grid_positions(case, lens):
    rows = []
    for n, keys, _ in lens:
        s = torch.arange(keys - n, keys, device="cuda", dtype=torch.int32)
        rows.append(torch.stack([s // (34 * 60), s // 60 % 34, s % 60], 1))
    return torch.cat(rows).contiguous()


def prepare(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    b, h, hk, d, page = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    lens = _lengths(case)
    per = -(-case["keys"] // page)
    pages = b * per + 3
    st = {"case": case, "lens": lens}
    st["k"], st["k_scales"] = _pages(case, pages, g, True)
    st["v"], st["v_scales"] = _pages(case, pages, g, False)
    st["table"] = torch.randperm(pages, generator=g, device="cuda")[: b * per].view(b, per).to(torch.int32)
    st["kv_lens"] = _int32([x[1] for x in lens])
    offsets = [0]
    for n, _, _ in lens:
        offsets.append(offsets[-1] + n)
    rows = offsets[-1]
    st["offsets"] = _int32(offsets)
    if case["op"] == "append":
        st["starts"] = _int32([x[1] - x[0] for x in lens])
        st["qkv"] = _randn((rows, (h + 2 * hk) * d), g, dt)
        st["qkv"][:, torch.randint(0, (h + 2 * hk) * d, (8,), generator=g, device="cuda")] *= 20.0
        st["wq"], st["wk"] = (0.5 + torch.rand(d, generator=g, device="cuda") for _ in range(2))
        st["positions"] = _grid_positions(case, lens) if case["axes"] == 3 else None
        st["q"] = torch.empty((rows, h, d), dtype=dt, device="cuda")
    elif case["op"] == "attention":
        st["q"] = _randn((rows, h, d), g, dt) * (0.5 + torch.rand(d, generator=g, device="cuda")).to(dt)
        if case["softcap"]:
            st["q"] *= 2.0  # scores that reach the cap's bend
        st["slopes"] = None
        if case["slopes"]:
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda", dtype=torch.float32) / h) * 0.5
        st["prefix"] = _int32([x[2] for x in lens]) if case["prefix"] else None
    if own:  # the handle of the same tensors that a program keeps
        from video_vae_decoder_qkv_gb300 import Cache

        st["cache"] = Cache(st["k"], st["v"], st["k_scales"], st["v_scales"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "read":
        return _own_read(state) if own else _plain_read(state)
    return _own_attention(state) if own else _plain_attention(state)


def _own_append(st):
    from video_vae_decoder_qkv_gb300 import cache_append, cache_read

    c = st["case"]
    q = cache_append(st["qkv"], st["wq"], st["wk"], st["cache"], st["table"], st["kv_lens"], q_offsets=st["offsets"],
                     positions=st["positions"], heads=c["heads"], rotary_dim=c["rotary"], out=st["q"])
    if c["cache"] != "e2m1":
        return {"q": q, "k": st["k"], "v": st["v"]}
    k, v = cache_read(st["cache"], st["table"], st["kv_lens"], starts=st["starts"], rows=c["rows"],
                      dtype=_DT[c["dtype"]])
    return {"q": q, "k": k, "v": v}


def _own_read(st):
    from video_vae_decoder_qkv_gb300 import cache_read

    c = st["case"]
    k, v = cache_read(st["cache"], st["table"], st["kv_lens"], rows=c["keys"], dtype=_DT[c["dtype"]])
    return {"k": k, "v": v}


def _own_attention(st):
    from video_vae_decoder_qkv_gb300 import cache_attention

    c = st["case"]
    out, lse = cache_attention(st["q"], st["cache"], st["table"], st["kv_lens"], q_offsets=st["offsets"],
                               max_rows=c["rows"], softcap=c["softcap"], slopes=st["slopes"], prefix_lens=st["prefix"])
    return {"out": out, "lse": lse}


def _item_of_rows(st, rows):
    """Every packed row's sequence and its position among that sequence's keys."""
    off = st["offsets"].long()
    r = torch.arange(rows, device="cuda")
    item = torch.bucketize(r, off[1:], right=True)
    return item, st["kv_lens"].long()[item] - (off[1:][item] - r)


def _normed(x, w):
    """x / rms(x) * w, with the squares summed in runs of 8 and the runs by halves, rounded to x's type."""
    d = x.shape[-1]
    f = x.float()
    s = (f * f).unflatten(-1, (d // 8, 8))
    total = s[..., 0]
    for i in range(1, 8):
        total = total + s[..., i]
    n = 1 << (d // 8 - 1).bit_length()
    total = torch.nn.functional.pad(total, (0, n - d // 8))
    while n > 1:
        n //= 2
        total = total[..., :n] + total[..., n:]
    inv = 1.0 / torch.sqrt(total / torch.full_like(total, d) + 1e-6)
    return ((f * inv) * w).to(x.dtype).float()


def _rotated(x, ang, dtype):
    """Pairs of the first channels turned by their angles (sine and cosine of binary64, rounded to binary32)."""
    r = 2 * ang.shape[-1]
    cos, sin = (f(ang.double()).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    u, v = x[..., 0:r:2], x[..., 1:r:2]
    turned = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1).to(dtype)


def _angles(case, positions):
    a, width = case["axes"], case["rotary"] // case["axes"]
    inv = torch.tensor([10000.0 ** (-2.0 * i / width) for i in range(width // 2)], dtype=torch.float32, device="cuda")
    return (positions.float().view(-1, a, 1) * inv).flatten(1)


def _plain_append(st):
    c = st["case"]
    rows, h, hk, d, dt = st["qkv"].shape[0], c["heads"], c["kv_heads"], c["dim"], _DT[c["dtype"]]
    item, pos = _item_of_rows(st, rows)
    ang = _angles(c, pos[:, None] if st["positions"] is None else st["positions"])
    x = st["qkv"].view(rows, h + 2 * hk, d)
    q = _rotated(_normed(x[:, :h], st["wq"]), ang, dt)
    k = _rotated(_normed(x[:, h:h + hk], st["wk"]), ang, dt)
    v = x[:, h + hk:]
    if c["cache"] != "e2m1":
        page, at = st["table"][item, pos // c["page"]].long(), pos % c["page"]
        st["k"][page, :, at] = k
        st["v"][page, :, at] = v
        return {"q": q, "k": st["k"], "v": st["v"]}
    kept = []
    for t in (k, v):
        code, scale = _e2m1(t.float().unflatten(-1, (-1, 16)))
        code = code.flatten(-2).to(torch.uint8)
        value = _value(code[..., 0::2] | (code[..., 1::2] << 4), scale.flatten(-2)).to(dt)
        dense = torch.zeros((c["batch"], c["rows"], hk, d), dtype=dt, device="cuda")
        dense[item, pos - st["starts"].long()[item]] = value
        kept.append(dense.transpose(1, 2).contiguous())
    return {"q": q, "k": kept[0], "v": kept[1]}


def _dense(st, which):
    """A cache's rows in order, binary32 [batch, kv_heads, keys, dim]."""
    c = st["case"]
    at = st["table"].long()
    t = st[which][at]
    t = t.float() if st[which + "_scales"] is None else _value(t, st[which + "_scales"].view(torch.uint8)[at].view(
        torch.float8_e4m3fn))
    return t.transpose(1, 2).reshape(c["batch"], c["kv_heads"], -1, c["dim"])[:, :, : c["keys"]]


def _plain_read(st):
    c = st["case"]
    there = torch.arange(c["keys"], device="cuda") < st["kv_lens"].view(-1, 1, 1)
    k, v = ((_dense(st, w) * there.unsqueeze(-1)).to(_DT[c["dtype"]]).contiguous() for w in ("k", "v"))
    return {"k": k, "v": v}


def _plain_attention(st):
    c = st["case"]
    b, h, hk, d, n, sk = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["rows"], c["keys"]
    rows, group, cap = st["q"].shape[0], h // hk, c["softcap"]
    item, pos = _item_of_rows(st, rows)
    lens = st["kv_lens"].long()
    within = torch.arange(rows, device="cuda") - st["offsets"].long()[item]
    q = torch.zeros((b, n, h, d), device="cuda")
    q[item, within] = st["q"].float()
    at = torch.full((b, n), -1, dtype=torch.int64, device="cuda")
    at[item, within] = pos
    q = q.view(b, n, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * n, d)
    j = torch.arange(sk, device="cuda")
    seen = j <= at.unsqueeze(-1)
    if st["prefix"] is not None:
        seen = seen | ((j < st["prefix"].view(-1, 1, 1)) & (at.unsqueeze(-1) >= 0))
    seen = seen & (j < lens.view(-1, 1, 1))
    s = (q @ _dense(st, "k").transpose(2, 3)).view(b, hk, group, n, sk)
    s *= 1.0 / math.sqrt(d)
    if cap:
        s = cap * torch.tanh(s / cap)
    if st["slopes"] is not None:
        s -= st["slopes"].view(1, hk, group, 1, 1) * (at.unsqueeze(-1) - j).abs().float().view(b, 1, 1, n, sk)
    s.masked_fill_(~seen.view(b, 1, 1, n, sk), -math.inf)
    top = s.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    del s
    total = p.sum(4, keepdim=True)
    lse = (top + torch.log(total)).view(b, h, n)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    o = (p.view(b, hk, group * n, sk) @ _dense(st, "v")).view(b, h, n, d)
    return {"out": o[item, :, within].to(st["q"].dtype), "lse": lse[item, :, within].t().contiguous()}


# --------------------------------------------------------------------------
# binary64, from the definitions
# --------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attention": _exact_attention}[case["op"]](st)


def _exact_rows(st, which, item, keys):
    """The first `keys` rows of a sequence, binary64 [kv_heads, keys, dim]."""
    page = st["case"]["page"]
    ids = st["table"][item, : -(-keys // page)].long()
    t = st[which][ids]
    if st[which + "_scales"] is None:
        t = t.double()
    else:
        lo, hi = t & 15, t >> 4
        code = torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=torch.float64, device="cuda")
        for half, x in ((0, lo), (1, hi)):
            e, m, sign = (x >> 1) & 3, x & 1, x >> 3
            mag = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0))
            code[..., half::2] = torch.where(sign == 1, -mag, mag)
        scale = st[which + "_scales"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
        t = code * scale.repeat_interleave(16, -1)
    return t.transpose(0, 1).reshape(t.shape[1], -1, t.shape[3])[:, :keys]


def _exact_append(st):
    c = st["case"]
    h, hk, d, r, page = c["heads"], c["kv_heads"], c["dim"], c["rotary"], c["page"]
    q, ks, vs, first = [], [], [], 0
    k_pool, v_pool = (None, None) if c["cache"] == "e2m1" else (st["k"].double(), st["v"].double())
    for item, (n, keys, _) in enumerate(st["lens"]):
        at = slice(first, first + n)
        first += n
        x = st["qkv"][at].view(n, h + 2 * hk, d).double()
        own_pos = torch.arange(keys - n, keys, device="cuda")
        # the angle is defined as a binary32 product; its sine and cosine are exact
        ang = _angles(c, own_pos[:, None] if st["positions"] is None else st["positions"][at]).double()
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]

        def done(t, w):
            y = t / torch.sqrt((t * t).mean(2, keepdim=True) + 1e-6) * w.double()
            if r:
                z = torch.view_as_complex(y[..., :r].reshape(n, -1, r // 2, 2).contiguous()) * turn
                y[..., :r] = torch.view_as_real(z).reshape(n, -1, r)
            return y

        q.append(done(x[:, :h], st["wq"]))
        if k_pool is not None:
            p, o = st["table"][item].long()[own_pos // page], own_pos % page
            k_pool[p, :, o] = done(x[:, h:h + hk], st["wk"])
            v_pool[p, :, o] = x[:, h + hk:]
    # what is rounded to 4 bits has no value of 64
    return {"q": torch.cat(q), "k": k_pool, "v": v_pool}


def _exact_read(st):
    c = st["case"]
    got = {}
    for w in ("k", "v"):
        t = torch.zeros(c["batch"], c["kv_heads"], c["keys"], c["dim"], dtype=torch.float64, device="cuda")
        for i, (_, keys, _) in enumerate(st["lens"]):
            t[i, :, :keys] = _exact_rows(st, w, i, keys)
        got[w] = t
    return got


def _exact_attention(st):
    c = st["case"]
    h, hk, d, cap = c["heads"], c["kv_heads"], c["dim"], c["softcap"]
    rows = st["q"].shape[0]
    out = torch.zeros(rows, h, d, dtype=torch.float64, device="cuda")
    lse = torch.full((h, rows), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for item, (n, keys, prefix) in enumerate(st["lens"]):
        if n == 0 or keys == 0:
            continue
        k, v = _exact_rows(st, "k", item, keys), _exact_rows(st, "v", item, keys)
        gap = (torch.arange(n, device="cuda") + keys - n)[:, None] - torch.arange(keys, device="cuda")
        hidden = (gap < 0) & ~(torch.arange(keys, device="cuda") < prefix)
        for head in range(h):
            s = (st["q"][first:first + n, head].double() @ k[head * hk // h].T) / math.sqrt(d)
            if cap:
                s = cap * torch.tanh(s / cap)
            if st["slopes"] is not None:
                s = s - float(st["slopes"][head]) * gap.abs()
            s = s.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(s, 1)
            out[first:first + n, head] = torch.exp(s - z[:, None]) @ v[head * hk // h]
            lse[head, first:first + n] = z
        first += n
    return {"out": out, "lse": lse}
