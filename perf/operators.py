"""Workloads of the attention block's operators: layer norm, the gradient of
the fused QK preparation, and attention (prompt, training step, single token).

``run`` computes an operator in its plain form (elementary torch operations in
binary32, rounded once at the end) or, with ``own`` set, through this
package's entry points; ``exact`` computes it in binary64 from its definition.
"""
import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_ESZ = {"fp16": 2, "bf16": 2, "fp32": 4}

# Most score elements and multiply-adds a drawn attention case may have (those
# of the largest listed one), so that the plain form's score matrix fits.
_MOST_SCORES = 40 * 8160 * 8160
_MOST_PAIR_DIMS = 40 * 8160 * 8160 * 128


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _attn(name, op, dtype, batch, heads, kv_heads, sq, sk, dim, *, causal=False, prefix=False, docs=0,
          ragged=False, softcap=0.0, slopes=False, layout="head", lens_seed=0):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "sq": sq, "sk": sk, "dim": dim, "causal": causal, "prefix": prefix, "docs": docs, "ragged": ragged,
            "softcap": softcap, "slopes": slopes, "layout": layout, "lens_seed": lens_seed}


def _ln(name, op, dtype, batch, rows, width, *, affine="shared"):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "rows": rows, "width": width, "affine": affine}


def _qk(name, dtype, batch, seq, heads, dim, rotary, axes, *, valid=None):
    return {"name": name, "op": "qk_grad", "dtype": dtype, "batch": batch, "seq": seq, "heads": heads, "dim": dim,
            "rotary": rotary, "axes": axes, "valid": seq if valid is None else valid}


def listed():
    return [
        # One token's norm before its projection while tokens are produced one by one: latency only.
        _ln("ln_token", "layer_norm", "fp16", 1, 1, 1024),
        # The norm of one 16x18x17-token decoder tile in a training step.
        _ln("ln_tile_train", "layer_norm_train", "fp16", 1, 4896, 1024),
        # Two packed clips of a large block with a weight and a bias of their own per clip
        # (an adaptive norm whose scale and shift come from the timestep), in a training step.
        _ln("ln_latent_train", "layer_norm_train", "bf16", 2, 65280, 5120, affine="batch"),
        # The smallest preparation (a 2x4x6 grid, four heads of 64): latency of a gradient.
        _qk("qk_grad_small", "fp16", 1, 48, 4, 64, 48, 3),
        # Eight decoder tiles in one call.
        _qk("qk_grad_tiles", "bf16", 8, 4896, 16, 64, 48, 3, valid=4890),
        # A latent grid of 16x34x60 tokens with forty heads of 128.
        _qk("qk_grad_latent", "bf16", 1, 32640, 40, 128, 96, 3),
        # Attention of one decoder tile: every token sees every token of the valid prefix.
        _attn("attn_tile", "attention", "fp16", 1, 16, 16, 4896, 4896, 64, ragged=True, lens_seed=3),
        # Four latent frames of 34x60 tokens, forty heads of 128, read token-major.
        _attn("attn_latent", "attention", "bf16", 1, 40, 40, 8160, 8160, 128, layout="token"),
        # A training step over packed clips: each attends within itself, causally after a prefix that
        # all of its tokens see; capped scores; eight K/V heads shared by forty.
        _attn("attn_clips_train", "attention_train", "bf16", 1, 40, 8, 6120, 6120, 128, causal=True, prefix=True,
              docs=5, softcap=30.0, lens_seed=4),
        # A training step of two decoder tiles with a bias that grows with distance.
        _attn("attn_tiles_train", "attention_train", "fp16", 2, 16, 16, 4896, 4896, 64, slopes=True, ragged=True,
              lens_seed=5),
        # One new token over one tile's cache: latency.
        _attn("attn_token", "attention", "fp16", 1, 16, 16, 1, 4896, 64, causal=True),
        # One new token for each of 32 requests over caches of uneven lengths, one slot idle.
        _attn("attn_token_batch", "attention", "bf16", 32, 40, 8, 1, 32768, 128, causal=True, ragged=True,
              lens_seed=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("layer_norm", "layer_norm_train", "qk_grad", "prompt", "train", "token"))
    if kind in ("layer_norm", "layer_norm_train"):
        width = _log(rng, 64, 8192)
        rows = _log(rng, 1, min(65280, 65280 * 5120 // width))
        batch = rng.choice((1, 1, 2, 3))
        rows = max(batch, rows // batch * batch)
        c = _ln(None, kind, rng.choice(("fp16", "bf16", "fp32")), batch, rows, width,
                affine=rng.choice(("shared", "batch", "none")))
    elif kind == "qk_grad":
        dim = rng.choice((32, 48, 64, 80, 96, 128))
        heads = rng.randint(1, 40)
        axes = rng.choice((1, 3))
        rotary = dim if axes == 1 else dim // 8 * 6 // 6 * 6
        batch = rng.choice((1, 1, 2, 4))
        seq = _log(rng, 1, max(1, 32640 * 40 * 128 // (heads * dim * batch)))
        c = _qk(None, rng.choice(("fp16", "bf16")), batch, min(seq, 65280), heads, dim, rotary, axes)
        c["valid"] = c["seq"] - rng.randint(0, c["seq"] // 8)
    else:
        dim = rng.choice((40, 64, 64, 72, 96, 128, 128))
        kv = rng.choice((1, 2, 4, 8, 12, 16))
        heads = kv * rng.choice((1, 1, 2, 5))
        heads = min(heads, 40) // kv * kv
        dtype = rng.choice(("fp16", "bf16"))
        cap = rng.choice((0.0, 0.0, 20.0, 50.0))
        slopes = rng.random() < 0.3
        seed = rng.randrange(1 << 20)
        if kind == "token":
            batch = _log(rng, 1, 48)
            sk = _log(rng, 1, min(65536, 32 * 40 * 32768 // (batch * heads)))
            c = _attn(None, "attention", dtype, batch, heads, kv, min(sk, rng.choice((1, 1, 2, 4))), sk, dim,
                      causal=True, ragged=rng.random() < 0.7, softcap=cap, slopes=slopes, lens_seed=seed)
        else:
            docs = rng.choice((0, 0, 3, 9))
            batch = 1 if docs else rng.choice((1, 1, 2, 3))
            most = math.sqrt(min(_MOST_SCORES, _MOST_PAIR_DIMS / dim) / (batch * heads) / (4 if kind == "train" else 1))
            s = _log(rng, 17, min(most, 16384))
            causal = rng.random() < 0.5
            c = _attn(None, "attention_train" if kind == "train" else "attention", dtype, batch, heads, kv, s, s, dim,
                      causal=causal, prefix=causal and rng.random() < 0.5, docs=docs,
                      ragged=not docs and rng.random() < 0.5, softcap=cap, slopes=slopes,
                      layout=rng.choice(("head", "token")), lens_seed=seed)
    del c["name"]
    return c


def _lengths(case):
    """What the case's lens_seed says of lengths: (q_lens, kv_lens, doc_offsets, prefix_lens) as lists, or None each."""
    r = random.Random(case["lens_seed"])
    b, sq, sk = case["batch"], case["sq"], case["sk"]
    q_lens = kv_lens = docs = prefix = None
    if case["docs"]:
        cuts = sorted(r.randint(0, sq) for _ in range(case["docs"] - 1))
        docs = [0] + cuts + [sq - r.randint(0, sq // 50)]
        docs[-1] = max(docs[-1], docs[-2])
    elif case["ragged"]:
        if sq == sk:
            kv_lens = [sk - r.randint(0, sk // 16) for _ in range(b)]
            q_lens = list(kv_lens)
        else:
            kv_lens = [max(sq, int(sk * r.uniform(0.25, 1.0))) for _ in range(b)]
            if b > 4:
                kv_lens[r.randrange(b)] = 0
    if case["prefix"]:
        n = case["docs"] or b
        longest = [docs[i + 1] - docs[i] for i in range(n)] if docs else (kv_lens or [sk] * b)
        prefix = [r.randint(0, max(0, x // 3)) for x in longest]
    return q_lens, kv_lens, docs, prefix


def _segments(case):
    """(item, first row, rows, keys, position of the first row, prefix) of every stretch of rows that shares its keys."""
    q_lens, kv_lens, docs, prefix = _lengths(case)
    if docs:
        return [(0, docs[i], docs[i + 1] - docs[i], docs[i + 1] - docs[i], 0, prefix[i] if prefix else 0)
                for i in range(len(docs) - 1)]
    got = []
    for i in range(case["batch"]):
        n = q_lens[i] if q_lens else case["sq"]
        keys = kv_lens[i] if kv_lens else case["sk"]
        got.append((i, 0, n, keys, 0 if case["sq"] == case["sk"] else keys - n, prefix[i] if prefix else 0))
    return got


def _pairs(case):
    """Visible (query, key) pairs of one head, over the whole batch."""
    total = 0
    for _, _, n, keys, start, prefix in _segments(case):
        if not case["causal"]:
            total += n * keys
        else:
            for i in range(n):
                total += max(0, min(keys, max(prefix, start + i + 1)))
    return total


def work(case):
    op = case["op"]
    if op in ("layer_norm", "layer_norm_train"):
        n, e = case["rows"] * case["width"], _ESZ[case["dtype"]]
        w = {"none": 0, "shared": 1, "batch": case["batch"]}[case["affine"]] * case["width"] * 8
        if op == "layer_norm":
            return {"bytes": 2 * n * e + w + 8 * case["rows"], "flops": 8 * n}
        # x, dy in; y, dx out (what stays on the chip between the two passes is not counted)
        return {"bytes": 4 * n * e + 2 * w + 8 * case["rows"], "flops": 20 * n}
    if op == "qk_grad":
        n = case["batch"] * case["valid"] * case["heads"] * case["dim"]
        every = case["batch"] * case["seq"] * case["heads"] * case["dim"]
        # q and k of the packed rows, three gradients in; the packed gradient out
        return {"bytes": 2 * (2 * n + 3 * n + 3 * every) + 4 * case["batch"] * case["seq"] * case["axes"] + 16 * case["dim"],
                "flops": 2 * n * 20}
    d, e, h = case["dim"], _ESZ[case["dtype"]], case["heads"]
    q = sum(x[2] for x in _segments(case)) * h * d * e
    kv = 2 * sum(x[3] for x in _segments(case)) * case["kv_heads"] * d * e
    rows = case["batch"] * case["sq"] * h
    pairs = _pairs(case) * h
    if op == "attention":
        return {"bytes": q + kv + rows * d * e + 4 * rows, "flops": 4 * d * pairs}
    # q, k, v, dout in; out, lse, dq, dk, dv out
    out = rows * d * e
    every = 2 * case["batch"] * case["sk"] * case["kv_heads"] * d * e
    return {"bytes": 2 * q + kv + 2 * out + 4 * rows + every, "flops": 14 * d * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFFFFFF)


def _randn(shape, g, dtype):
    # 16-bit draws directly: a binary32 copy of the largest inputs is not needed
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _outliers(t, g, factor):
    """A thousandth of the columns carry larger values in every row, as activations do."""
    n = max(1, t.shape[-1] // 1000)
    cols = torch.randint(0, t.shape[-1], (n,), generator=g, device="cuda")
    t[..., cols] *= factor
    return t


def _int32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def _grid_positions(case):
    s = torch.arange(case["seq"], device="cuda", dtype=torch.int64)
    if case["axes"] == 1:
        p = s[:, None]
    else:
        wide = max(1, min(60, int(math.isqrt(case["seq"]))))
        high = max(1, min(34, case["seq"] // wide))
        p = torch.stack([s // (high * wide), s // wide % high, s % wide], 1)
    return p.to(torch.int32).repeat(case["batch"], 1).contiguous()


def prepare(case, seed):
    g, dt, op = _gen(seed), _DT[case["dtype"]], case["op"]
    st = {"case": case}
    if op in ("layer_norm", "layer_norm_train"):
        rows, c, b = case["rows"], case["width"], case["batch"]
        st["x"] = _outliers(_randn((rows, c), g, dt), g, 20.0)
        st["x"] += 0.5
        shape = (c,) if case["affine"] == "shared" else (b, c)
        st["weight"] = st["bias"] = None
        if case["affine"] != "none":
            st["weight"] = 1.0 + 0.2 * _randn(shape, g, torch.float32)
            st["bias"] = 0.1 * _randn(shape, g, torch.float32)
        if op == "layer_norm_train":
            st["dy"] = _randn((rows, c), g, dt)
        return st
    if op == "qk_grad":
        b, s, h, d = case["batch"], case["seq"], case["heads"], case["dim"]
        st["qkv"] = _outliers(_randn((b * s, 3 * h * d), g, dt), g, 30.0)
        st["wq"] = 0.5 + torch.rand(d, generator=g, device="cuda")
        st["wk"] = 0.5 + torch.rand(d, generator=g, device="cuda")
        st["positions"] = _grid_positions(case)
        st["dq"], st["dk"], st["dv"] = (_randn((b, h, s, d), g, dt) for _ in range(3))
        return st
    b, h, hk, sq, sk, d = (case[k] for k in ("batch", "heads", "kv_heads", "sq", "sk", "dim"))

    def heads(n, s, normed):
        shape = (b, n, s, d) if case["layout"] == "head" else (b, s, n, d)
        t = _randn(shape, g, dt)
        if normed:  # Q and K come out of a per-head RMS norm with a weight
            t *= (0.5 + torch.rand(d, generator=g, device="cuda")).to(dt)
            if case["softcap"]:
                t *= 2.0  # scores that reach the cap's bend
        else:
            _outliers(t, g, 10.0)
        return t if case["layout"] == "head" else t.transpose(1, 2)

    st["q"], st["k"], st["v"] = heads(h, sq, True), heads(hk, sk, True), heads(hk, sk, False)
    if op == "attention_train":
        st["dout"] = _randn((b, h, sq, d), g, dt)
    q_lens, kv_lens, docs, prefix = _lengths(case)
    st["q_lens"], st["kv_lens"], st["doc_offsets"], st["prefix_lens"] = (_int32(v) for v in (q_lens, kv_lens, docs, prefix))
    st["slopes"] = None
    if case["slopes"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda", dtype=torch.float32) / h) * 0.5
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op in ("layer_norm", "layer_norm_train"):
        return _own_layer_norm(state) if own else _plain_layer_norm(state)
    if op == "qk_grad":
        return _own_qk_grad(state) if own else _plain_qk_grad(state)
    return _own_attention(state) if own else _plain_attention(state)


def _own_layer_norm(st):
    from video_vae_decoder_qkv_gb300 import layer_norm, layer_norm_backward

    batch = st["case"]["batch"]
    y, stats = layer_norm(st["x"], st["weight"], st["bias"], eps=1e-6, batch=batch)
    if "dy" not in st:
        return {"y": y, "stats": stats}
    dx, dw, db = layer_norm_backward(st["dy"], st["x"], st["weight"], stats, batch=batch)
    return {"y": y, "stats": stats, "dx": dx, "dw": dw, "db": db}


def _own_qk_grad(st):
    from video_vae_decoder_qkv_gb300 import prepare_backward

    c = st["case"]
    dqkv, dwq, dwk = prepare_backward(st["dq"], st["dk"], st["dv"], st["qkv"], st["wq"], st["wk"], st["positions"],
                                      heads=c["heads"], head_dim=c["dim"], rotary_dim=c["rotary"], batch=c["batch"],
                                      valid_len=c["valid"])
    return {"dqkv": dqkv, "dwq": dwq, "dwk": dwk}


def _own_attention(st):
    from video_vae_decoder_qkv_gb300 import attention, attention_backward

    c = st["case"]
    kw = dict(softcap=c["softcap"], slopes=st["slopes"], causal=c["causal"], prefix_lens=st["prefix_lens"],
              doc_offsets=st["doc_offsets"], q_lens=st["q_lens"], kv_lens=st["kv_lens"])
    out, lse = attention(st["q"], st["k"], st["v"], **kw)
    if "dout" not in st:
        return {"out": out, "lse": lse}
    dq, dk, dv = attention_backward(st["dout"], st["q"], st["k"], st["v"], out, lse, **kw)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _plain_layer_norm(st):
    x, c = st["x"].float(), st["case"]
    b, w = c["batch"], c["width"]
    x = x.view(b, -1, w)
    mean = x.mean(2, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(2, keepdim=True) + 1e-6)
    xh = (x - mean) * rstd
    weight = bias = None
    if st["weight"] is not None:
        weight, bias = st["weight"].view(-1, 1, w), st["bias"].view(-1, 1, w)
    y = xh if weight is None else xh * weight + bias
    got = {"y": y.to(st["x"].dtype).view(-1, w), "stats": torch.cat([mean, rstd], 2).view(-1, 2)}
    if "dy" not in st:
        return got
    del y
    dy = st["dy"].float().view(b, -1, w)
    g = dy if weight is None else dy * weight
    dx = rstd * (g - g.mean(2, keepdim=True) - xh * (g * xh).mean(2, keepdim=True))
    got["dx"] = dx.to(st["x"].dtype).view(-1, w)
    got["dw"] = got["db"] = None
    if weight is not None:
        dw, db = (dy * xh).sum(1), dy.sum(1)
        got["dw"] = (dw if c["affine"] == "batch" else dw.sum(0)).view_as(st["weight"])
        got["db"] = (db if c["affine"] == "batch" else db.sum(0)).view_as(st["weight"])
    return got


def _angles(case, positions):
    """Angles of each row's rotary pairs, binary32 [rows, rotary/2]: the position times the pair's inverse frequency
    (rounded to binary32), axis after axis."""
    a, width = case["axes"], case["rotary"] // case["axes"]
    inv = torch.tensor([10000.0 ** (-2.0 * i / width) for i in range(width // 2)], dtype=torch.float32,
                       device=positions.device)
    return (positions.float().view(-1, a, 1) * inv).view(positions.shape[0], -1)


def _plain_qk_grad(st):
    c = st["case"]
    b, s, h, d, r = (c[k] for k in ("batch", "seq", "heads", "dim", "rotary"))
    ang = _angles(c, st["positions"]).view(b, s, 1, r // 2)
    cos, sin = torch.cos(ang), torch.sin(ang)
    keep = (torch.arange(s, device="cuda") < c["valid"]).view(1, s, 1, 1)
    x = st["qkv"].view(b, s, 3, h, d)

    def one(xt, w, dy):
        xt, dy = xt.float(), dy.transpose(1, 2).float() * keep
        inv = 1.0 / torch.sqrt(xt.square().mean(3, keepdim=True) + 1e-6)
        du, dv = dy[..., 0:r:2], dy[..., 1:r:2]
        dn = dy.clone()
        dn[..., 0:r:2] = du * cos + dv * sin
        dn[..., 1:r:2] = dv * cos - du * sin
        xh = xt * inv
        dw = (dn * xh).sum((0, 1, 2))
        g = dn * w
        return inv * (g - xh * (g * xh).mean(3, keepdim=True)), dw

    dqkv = torch.empty_like(x)
    dqkv[:, :, 0], dwq = one(x[:, :, 0], st["wq"], st["dq"])
    dqkv[:, :, 1], dwk = one(x[:, :, 1], st["wk"], st["dk"])
    dqkv[:, :, 2] = st["dv"].transpose(1, 2) * keep
    return {"dqkv": dqkv.view(b * s, 3 * h * d), "dwq": dwq, "dwk": dwk}


def _visible(st):
    """Which keys each row sees, [batch, sq, sk], and the distance |row's position - key's position|."""
    c = st["case"]
    sq, sk = c["sq"], c["sk"]
    i = torch.arange(sq, device="cuda").view(1, sq, 1)
    j = torch.arange(sk, device="cuda").view(1, 1, sk)
    if st["doc_offsets"] is not None:
        off = st["doc_offsets"].long()
        doc = torch.bucketize(torch.arange(sq, device="cuda"), off, right=True) - 1
        inside = doc < off.numel() - 1
        doc = doc.clamp(max=off.numel() - 2)
        first = off[doc]
        vis = (doc.view(1, sq, 1) == doc.view(1, 1, sk)) & inside.view(1, sq, 1) & inside.view(1, 1, sk)
        i, j = i - first.view(1, sq, 1), j - first.view(1, 1, sk)
        prefix = None if st["prefix_lens"] is None else st["prefix_lens"].long()[doc].view(1, sq, 1)
    else:
        whole = torch.full((c["batch"],), 1, device="cuda", dtype=torch.int64)
        ql = (sq * whole if st["q_lens"] is None else st["q_lens"].long()).view(-1, 1, 1)
        kl = (sk * whole if st["kv_lens"] is None else st["kv_lens"].long()).view(-1, 1, 1)
        vis = (i < ql) & (j < kl)
        if sq != sk:
            i = i + kl - ql
        prefix = None if st["prefix_lens"] is None else st["prefix_lens"].long().view(-1, 1, 1)
    if c["causal"]:
        seen = j <= i
        if prefix is not None:
            seen = seen | (j < prefix)
        vis = vis & seen
    return vis, (i - j).abs()


def _plain_attention(st):
    c = st["case"]
    b, h, hk, sq, sk, d = (c[k] for k in ("batch", "heads", "kv_heads", "sq", "sk", "dim"))
    n, scale, cap = h // hk, 1.0 / math.sqrt(c["dim"]), c["softcap"]
    q = st["q"].float().reshape(b, hk, n * sq, d)
    k, v = st["k"].float(), st["v"].float()
    vis, dist = _visible(st)
    s = (q @ k.transpose(2, 3)).view(b, hk, n, sq, sk)
    s *= scale
    bend = None
    if cap:
        s = torch.tanh(s / cap)
        bend = 1.0 - s * s if "dout" in st else None
        s *= cap
    if st["slopes"] is not None:
        s -= st["slopes"].view(1, hk, n, 1, 1) * dist.view(-1, 1, 1, sq, sk).float()
    s.masked_fill_(~vis.view(-1, 1, 1, sq, sk), -math.inf)
    top = s.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    del s
    total = p.sum(4, keepdim=True)
    lse = (top + torch.log(total)).view(b, h, sq)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    p = p.view(b, hk, n * sq, sk)
    o = p @ v
    got = {"out": o.view(b, h, sq, d).to(st["q"].dtype), "lse": lse}
    if "dout" not in st:
        return got
    do = st["dout"].float().reshape(b, hk, n * sq, d)
    delta = (do * o).sum(3, keepdim=True)
    got["dv"] = (p.transpose(2, 3) @ do).to(st["v"].dtype)
    ds = do @ v.transpose(2, 3)
    ds -= delta
    ds *= p
    del p
    if bend is not None:
        ds *= bend.view_as(ds)
    ds *= scale
    got["dq"] = (ds @ k).view(b, h, sq, d).to(st["q"].dtype)
    got["dk"] = (ds.transpose(2, 3) @ q).to(st["k"].dtype)
    return got


# --------------------------------------------------------------------------
# binary64, from the definitions
# --------------------------------------------------------------------------

def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("layer_norm", "layer_norm_train"):
        return _exact_layer_norm(st)
    if op == "qk_grad":
        return _exact_qk_grad(st)
    return _exact_attention(st)


def _exact_layer_norm(st):
    c = st["case"]
    b, per, w = c["batch"], c["rows"] // c["batch"], c["width"]
    y = torch.empty(c["rows"], w, dtype=torch.float64, device="cuda")
    dx = torch.empty_like(y) if "dy" in st else None
    stats = torch.empty(c["rows"], 2, dtype=torch.float64, device="cuda")
    dw = torch.zeros(b, w, dtype=torch.float64, device="cuda")
    db = torch.zeros_like(dw)
    for item in range(b):
        gamma = beta = None
        if st["weight"] is not None:
            at = item if c["affine"] == "batch" else 0
            gamma, beta = st["weight"].reshape(-1, w)[at].double(), st["bias"].reshape(-1, w)[at].double()
        for r0 in range(item * per, (item + 1) * per, 4096):
            r1 = min(r0 + 4096, (item + 1) * per)
            x = st["x"][r0:r1].double()
            mu = x.sum(1) / w
            dev = x - mu[:, None]
            sd = torch.sqrt((dev * dev).sum(1) / w + 1e-6)
            xh = dev / sd[:, None]
            stats[r0:r1, 0], stats[r0:r1, 1] = mu, 1.0 / sd
            y[r0:r1] = xh if gamma is None else xh * gamma + beta
            if dx is not None:
                dy = st["dy"][r0:r1].double()
                dw[item] += (dy * xh).sum(0)
                db[item] += dy.sum(0)
                g = dy if gamma is None else dy * gamma
                a, e = g.sum(1) / w, (g * xh).sum(1) / w
                dx[r0:r1] = (g - a[:, None] - xh * e[:, None]) / sd[:, None]
    if dx is None:
        return {"y": y, "stats": stats}
    got = {"y": y, "stats": stats, "dx": dx, "dw": None, "db": None}
    if st["weight"] is not None:
        got["dw"], got["db"] = (dw, db) if c["affine"] == "batch" else (dw.sum(0), db.sum(0))
    return got


def _exact_qk_grad(st):
    c = st["case"]
    b, s, h, d, r = (c[k] for k in ("batch", "seq", "heads", "dim", "rotary"))
    dqkv = torch.zeros(b * s, 3, h, d, dtype=torch.float32 if b * s * h * d > 1 << 27 else torch.float64, device="cuda")
    dws = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)]
    for item in range(b):
        for s0 in range(0, c["valid"], 2048):
            s1 = min(s0 + 2048, c["valid"])
            rows = slice(item * s + s0, item * s + s1)
            # the angle is defined as a binary32 product; its sine and cosine are exact
            ang = _angles(c, st["positions"][rows]).double()[:, None, :]
            turn = torch.complex(torch.cos(ang), torch.sin(ang))
            for t, (w, dy) in enumerate(((st["wq"], st["dq"]), (st["wk"], st["dk"]))):
                x = st["qkv"][rows].view(s1 - s0, 3, h, d)[:, t].double()
                dn = dy[item, :, s0:s1].transpose(0, 1).double().contiguous()
                if r:
                    z = torch.view_as_complex(dn[..., :r].reshape(s1 - s0, h, r // 2, 2)) * turn.conj()
                    dn[..., :r] = torch.view_as_real(z).reshape(s1 - s0, h, r)
                ms = (x * x).sum(2, keepdim=True) / d + 1e-6
                g = dn * w.double()
                dqkv[rows, t] = (g / ms.sqrt() - x * (g * x).sum(2, keepdim=True) / (d * ms * ms.sqrt())).to(dqkv.dtype)
                dws[t] += (dn * x / ms.sqrt()).sum((0, 1))
            dqkv[rows, 2] = st["dv"][item, :, s0:s1].transpose(0, 1).to(dqkv.dtype)
    return {"dqkv": dqkv.view(b * s, 3 * h * d), "dwq": dws[0], "dwk": dws[1]}


def _exact_attention(st):
    c = st["case"]
    b, h, hk, sq, sk, d = (c[k] for k in ("batch", "heads", "kv_heads", "sq", "sk", "dim"))
    n, cap, train = h // hk, c["softcap"], "dout" in st
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(b, h, sq, d, **f64), torch.full((b, h, sq), -math.inf, **f64)
    dq = dk = dv = None
    if train:
        dq, dk, dv = torch.zeros(b, h, sq, d, **f64), torch.zeros(b, hk, sk, d, **f64), torch.zeros(b, hk, sk, d, **f64)
    for item, first, rows, keys, start, prefix in _segments(c):
        if rows <= 0 or keys <= 0:
            continue
        # in a packed sequence the keys of a document are its own rows
        k0 = first if c["docs"] else 0
        for head in range(h):
            kv = head // n
            k, v = st["k"][item, kv, k0:k0 + keys].double(), st["v"][item, kv, k0:k0 + keys].double()
            for r0 in range(0, rows, 4096):
                r1 = min(r0 + 4096, rows)
                at = slice(first + r0, first + r1)
                q = st["q"][item, head, at].double()
                s = (q @ k.T) / math.sqrt(d)
                if cap:
                    s = cap * torch.tanh(s / cap)
                if st["slopes"] is not None or c["causal"]:
                    gap = (torch.arange(r0, r1, device="cuda") + start)[:, None] - torch.arange(keys, device="cuda")
                capped = s
                if st["slopes"] is not None:
                    s = s - float(st["slopes"][head]) * gap.abs()
                if c["causal"]:
                    s = torch.where((gap >= 0) | (torch.arange(keys, device="cuda") < prefix), s, -math.inf)
                z = torch.logsumexp(s, 1)
                p = torch.where(torch.isneginf(z)[:, None], 0.0, torch.exp(s - z[:, None]))
                o = p @ v
                out[item, head, at], lse[item, head, at] = o, z
                if train:
                    do = st["dout"][item, head, at].double()
                    dv[item, kv, k0:k0 + keys] += p.T @ do
                    ds = p * (do @ v.T - (do * o).sum(1, keepdim=True)) / math.sqrt(d)
                    if cap:
                        ds = ds * (1.0 - (capped / cap) ** 2)
                    dq[item, head, at] = ds @ k
                    dk[item, kv, k0:k0 + keys] += ds.T @ q
    got = {"out": out, "lse": lse}
    if train:
        got.update(dq=dq, dk=dk, dv=dv)
    return got
