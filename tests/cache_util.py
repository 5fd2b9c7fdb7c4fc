"""Paged caches for the tests, with what they stand for in binary64, and the
plain form of the 4-bit format."""
import math

import block_util as bu
import torch

from video_vae_decoder_qkv_gb300 import Cache

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def code_values(codes):
    """What nibbles 0..15 stand for, in binary64."""
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=codes.device)
    return table[codes.long()]


def encode(y, tensor_scale=1.0):
    """(codes, scale bytes) of rows y [..., dim] in a 16-bit type: nibbles [..., dim] and e4m3 bytes [..., dim / 16].

    The format's own steps: each is one binary32 operation, rounded once, as the header states them."""
    g = y.float().unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    to_scale = torch.tensor(1.0 / (6.0 * tensor_scale), dtype=torch.float64).float().to(y.device)
    scale = (top * to_scale).clamp(2.0 ** -9, 448.0)
    finite = torch.isfinite(g).all(-1)
    scale = torch.where(finite, scale, 1.0).to(torch.float8_e4m3fn)
    factor = 1.0 / (scale.float() * torch.full_like(top, tensor_scale))
    z = g * factor.unsqueeze(-1)
    # the nearest value, the even code where two are as near
    a, at = z.abs().double().clamp(max=6.0), torch.tensor(VALUES, dtype=torch.float64, device=y.device)
    off = (a.unsqueeze(-1) - at).abs()
    code = off.argmin(-1)
    tie = (code < 7) & (off.gather(-1, code.unsqueeze(-1)) == off.gather(-1, (code + 1).clamp(max=7).unsqueeze(-1))).squeeze(-1)
    code = torch.where(tie & (code % 2 == 1), code + 1, code)
    code = code + 8 * (torch.signbit(z)).long()
    code = torch.where(finite.unsqueeze(-1), code, 0)
    bytes_ = torch.where(finite, scale.view(torch.uint8), torch.full_like(scale.view(torch.uint8), 0x7F))
    return code.flatten(-2).to(torch.uint8), bytes_


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def values(cache):
    """(k, v) of all pages in binary64 [pages, kv_heads, page_size, dim]."""
    if cache.dtype != "e2m1":
        return cache.k.double(), cache.v.double()
    out = []
    for t, s, ts in ((cache.k, cache.k_scales, cache.k_scale), (cache.v, cache.v_scales, cache.v_scale)):
        wide = s.double().repeat_interleave(16, -1)
        out.append(code_values(unpack(t)) * wide * float(torch.tensor(ts).float()))
    return tuple(out)


def rows_of(pool, table, keys):
    """A sequence's rows in order [kv_heads, keys, dim]; pages outside the pool are zeros."""
    n, heads, page, dim = pool.shape
    got = torch.zeros(heads, keys, dim, dtype=pool.dtype, device=pool.device)
    for i in range((keys + page - 1) // page):
        at = int(table[i]) if i < len(table) else -1
        if 0 <= at < n:
            m = min(page, keys - i * page)
            got[:, i * page:i * page + m] = pool[at, :, :m]
    return got


def build(lens, kv_heads, dim, page, fmt, *, seed=0, layout="head", k_scale=1.0, v_scale=1.0, spare=2, extra_pages=0):
    """(cache, table, kv_lens): random rows for the sequences, NaN wherever no sequence has a row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = max(1, max((k + page - 1) // page for k in lens)) + extra_pages
    pages = len(lens) * per + spare
    table = torch.randperm(pages, generator=g, device="cuda")[:len(lens) * per].view(len(lens), per).int()
    k, v = (torch.randn(pages, kv_heads, page, dim, generator=g, device="cuda") for _ in range(2))
    v[..., 0] *= 6.0
    written = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        written[table[b].long()[at // page], at % page] = True
    hole = ~written[:, None, :, None].expand(pages, kv_heads, page, dim)
    if fmt == "e2m1":
        parts, scales = [], []
        for t, s in ((k, k_scale), (v, v_scale)):
            c, b = encode((t * s).bfloat16(), s)
            b[hole[..., : dim // 16]] = 0x7F
            parts.append(pack(c))
            scales.append(b.view(torch.float8_e4m3fn))
        cache = Cache(*parts, *scales, k_scale=k_scale, v_scale=v_scale)
    else:
        k, v = (t.to(fmt).masked_fill(hole, math.nan) for t in (k, v))
        if layout == "row":  # [pages, page, kv_heads, dim], K and V beside each other
            both = torch.empty(pages, 2, page, kv_heads, dim, dtype=fmt, device="cuda")
            both[:, 0], both[:, 1] = k.transpose(1, 2), v.transpose(1, 2)
            k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
        cache = Cache(k, v)
    return cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def attention(q, cache, table, lens, offsets, *, causal=True, prefix=None, scale=None, softcap=0.0, slopes=None):
    """Plain attention in binary64, sequence by sequence: {"out", "lse" and their bounds}, [tokens, heads, ...]."""
    k_all, v_all = values(cache)
    tokens, heads, dim = q.shape
    out = {n: torch.zeros(tokens, heads, dim, dtype=torch.float64, device="cuda") for n in ("out", "out_bound")}
    for n in ("lse", "lse_bound"):
        out[n] = torch.zeros(tokens, heads, dtype=torch.float64, device="cuda")
    owned = torch.zeros(tokens, dtype=torch.bool)
    for b, keys in enumerate(lens):
        r0, r1 = offsets[b], offsets[b + 1]
        if r1 <= r0:
            continue
        owned[r0:r1] = True
        if keys <= 0:
            out["lse"][r0:r1] = -math.inf
            continue
        k, v = rows_of(k_all, table[b], keys), rows_of(v_all, table[b], keys)
        vis, dist = bu.visible(r1 - r0, keys, 1, causal, None if prefix is None else [prefix[b]],
                               q_starts=[keys - (r1 - r0)])
        got = bu.attention(q[r0:r1].transpose(0, 1)[None], k[None], v[None], vis, dist, scale=scale, softcap=softcap,
                           slopes=slopes)
        if cache.dtype == "e2m1" or q.dtype == torch.float16:
            # P is binary16, raised so that the row's largest is at least 2^7: a value below 2^-14 is off by up to half of
            # binary16's smallest step, 2^-25, which is 2^-32 of the largest, and the row's sum is no smaller than that
            seen = vis[0].any(0)[None, :, None]
            far = vis.double() @ torch.where(seen, v, 0.0).abs()
            got["out_bound"] += 2.0 ** -32 * far.repeat_interleave(heads // cache.kv_heads, 0)[None]
        for n in ("out", "out_bound"):
            out[n][r0:r1] = got[n][0].transpose(0, 1)
        for n in ("lse", "lse_bound"):
            out[n][r0:r1] = got[n][0].transpose(0, 1)
    return out, owned
