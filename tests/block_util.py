"""Plain binary64 forms of the attention block's operators, and the error
bounds their tests use."""
import math

import torch

# unit roundoff, and half the spacing of the smallest numbers, of each type
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
U32 = U[torch.float32]


def assert_within(got, want, bound, what):
    """|got - want| <= bound everywhere (want and bound in binary64)."""
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, off / bound.clamp(min=1e-300), torch.zeros_like(off)).reshape(-1)))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values are too far off; at {i}: "
                             f"{float(got.reshape(-1)[i])} for {float(want.reshape(-1)[i])} "
                             f"(bound {float(bound.reshape(-1)[i])})")


def assert_rel(got, want, most, what):
    """||got - want|| <= most ||want|| in the 2-norm."""
    off = float((got.double() - want).norm())
    norm = float(want.norm())
    assert off <= most * norm, f"{what}: off by {off:.3g} of {norm:.3g} ({off / max(norm, 1e-300):.3g}), {most:.3g} allowed"


def layer_norm(x, weight, bias, eps, batch):
    """(y, mean, rstd) in binary64; weight [C] or [batch, C]."""
    c = x.shape[1]
    x = x.double().reshape(batch, -1, c)
    mean = x.mean(2, keepdim=True)
    rstd = (((x - mean) ** 2).mean(2, keepdim=True) + eps) ** -0.5
    xh = (x - mean) * rstd
    w = 1.0 if weight is None else weight.double().reshape(-1, 1, c)
    b = 0.0 if bias is None else bias.double().reshape(-1, 1, c)
    return (xh * w + b).reshape(-1, c), mean.reshape(-1), rstd.reshape(-1)


def layer_norm_backward(dy, x, weight, eps, batch):
    """(dx, dw, db) in binary64, dw and db [batch, C] (per item)."""
    c = x.shape[1]
    _, mean, rstd = layer_norm(x, None, None, eps, 1)
    xh = ((x.double() - mean[:, None]) * rstd[:, None]).reshape(batch, -1, c)
    d = dy.double().reshape(batch, -1, c)
    g = d if weight is None else d * weight.double().reshape(-1, 1, c)
    dx = rstd.reshape(batch, -1, 1) * (g - g.mean(2, keepdim=True) - xh * (g * xh).mean(2, keepdim=True))
    return dx.reshape(-1, c), (d * xh).sum(1), d.sum(1)


def angles(positions, rotary, axis_dims, theta=10000.0):
    """The forward's angles: binary32 product of position and inverse frequency, in binary64."""
    cols = []
    for a, width in enumerate(axis_dims):
        inv = torch.tensor([theta ** (-2.0 * i / width) for i in range(width // 2)], dtype=torch.float32,
                           device=positions.device)
        cols.append(positions[:, a:a + 1].float() * inv)
    return torch.cat(cols, 1).double() if rotary else None


def norm_rope(x, w, ang, eps, rotary):
    """One of Q, K in binary64: x [rows, heads, D] -> rotated w x inv."""
    x = x.double()
    n = x * ((x * x).mean(2, keepdim=True) + eps) ** -0.5 * w.double()
    if rotary:
        z = torch.view_as_complex(n[..., :rotary].reshape(*n.shape[:2], rotary // 2, 2).contiguous())
        z = z * torch.polar(torch.ones_like(ang), ang)[:, None, :]
        n = torch.cat([torch.view_as_real(z).reshape(*n.shape[:2], rotary), n[..., rotary:]], 2)
    return n


def head_major(x, batch):
    """[tokens, heads, D] -> [batch, heads, S, D]."""
    return x.reshape(batch, -1, *x.shape[1:]).transpose(1, 2)


def visible(sq, sk, batch, causal=False, prefix_lens=None, doc_offsets=None, q_lens=None, kv_lens=None, q_starts=None,
            device="cuda"):
    """(who sees what [batch, sq, sk], |position - key| [batch, sq, sk]) from the definition, by plain loops."""
    vis = torch.zeros(batch, sq, sk, dtype=torch.bool)
    dist = torch.zeros(batch, sq, sk, dtype=torch.float64)
    runs = []
    if doc_offsets is not None:
        off = [int(x) for x in doc_offsets]
        for d in range(len(off) - 1):
            runs.append((0, off[d], off[d], off[d + 1] - off[d], off[d + 1] - off[d], 0,
                         int(prefix_lens[d]) if prefix_lens is not None else 0))
    else:
        for b in range(batch):
            n = sq if q_lens is None else min(max(int(q_lens[b]), 0), sq)
            keys = sk if kv_lens is None else min(max(int(kv_lens[b]), 0), sk)
            start = int(q_starts[b]) if q_starts is not None else (0 if sq == sk else keys - n)
            runs.append((b, 0, 0, n, keys, start, int(prefix_lens[b]) if prefix_lens is not None else 0))
    for b, r0, k0, n, keys, start, prefix in runs:
        i = torch.arange(n)[:, None] + start
        j = torch.arange(keys)[None, :]
        see = torch.ones(n, keys, dtype=torch.bool)
        if causal:
            see = (j <= i) | (j < prefix)
        vis[b, r0:r0 + n, k0:k0 + keys] = see
        dist[b, r0:r0 + n, k0:k0 + keys] = (i - j).abs().double()
    return vis.to(device), dist.to(device)


def attention(q, k, v, vis, dist, dout=None, scale=None, softcap=0.0, slopes=None):
    """Attention in binary64: {"out", "lse", and with dout "dq", "dk", "dv"} and under "..._bound" how far the
    kernels' results may be from each.

    u is the type's unit roundoff.  A score is off by at most eps: the binary32 sum over D products, the hardware's
    2^x and the tanh built on it, together below 2^-20 (8 + scale sum|q||k| + softcap).  P (and dS) are rounded to
    the type before their products, so each term of a product's sum is off by 2 (u + eps) of itself; delta takes the
    rounded output; each result is rounded once."""
    group = q.shape[1] // k.shape[1]
    u, tiny = U[q.dtype], TINY[q.dtype]
    scale = q.shape[3] ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    seen = vis.any(1)[:, None, :, None]  # values that nobody sees may be anything
    k, v = torch.where(seen, k, 0.0), torch.where(seen, v, 0.0)
    rows = vis.any(2)[:, None, :, None]
    q = torch.where(rows, q, 0.0)
    kk, vv = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    mask = vis[:, None]
    z = scale * (q @ kk.transpose(2, 3))
    terms = scale * (q.abs() @ kk.abs().transpose(2, 3))
    t = torch.tanh(z / softcap) if softcap else None
    s = softcap * t if softcap else z
    if slopes is not None:
        s = s - slopes.double().view(1, -1, 1, 1) * dist[:, None]
        terms = terms + slopes.double().abs().view(1, -1, 1, 1) * dist[:, None]
    s = s.masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, 3)
    p = torch.where(mask, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    eps = 2.0 ** -20 * (8 + softcap + torch.where(mask, terms, 0.0).amax(3, keepdim=True))
    out = p @ vv
    got = {"out": out, "lse": lse}
    got["out_bound"] = u * out.abs() + tiny + 2 * (u + eps) * (p @ vv.abs()) + 1e-12
    got["lse_bound"] = torch.where(lse.isinf(), 0.0, 2 * eps[..., 0] + 2.0 ** -22 * lse.abs())
    if dout is None:
        return got
    do = torch.where(rows, dout.double(), 0.0)
    dp = do @ vv.transpose(2, 3)
    dp_terms = do.abs() @ vv.abs().transpose(2, 3)
    delta = (do * out).sum(3, keepdim=True)
    bend = (1 - t * t) if softcap else 1.0
    ds = p * (dp - delta) * bend
    o_terms = (do.abs() * (u * out.abs() + got["out_bound"])).sum(3, keepdim=True)
    ds_off = 2 * (u + eps) * ds.abs() + p * (2.0 ** -18 * (dp_terms + delta.abs()) + 2 * o_terms) + \
        (p * (dp - delta).abs() * 2.0 ** -18 if softcap else 0.0)
    # fp16's smallest numbers: dS below 2^-14 is held to an absolute 2^-25, P (kept 2^10 larger) to 2^-35
    if tiny > 1e-10:
        ds_off = ds_off + torch.where(mask, tiny, 0.0)
    fold = lambda x: x.view(x.shape[0], -1, group, *x.shape[2:]).sum(2)  # noqa: E731
    got["dq"] = scale * (ds @ kk)
    got["dk"] = scale * fold(ds.transpose(2, 3) @ q)
    got["dv"] = fold(p.transpose(2, 3) @ do)
    got["dq_bound"] = u * got["dq"].abs() + tiny + scale * (ds_off @ kk.abs()) + 1e-12
    got["dk_bound"] = u * got["dk"].abs() + tiny + scale * fold(ds_off.transpose(2, 3) @ q.abs()) + 1e-12
    p_off = 2 * (u + eps) * p + (torch.where(mask, 2.0 ** -34, 0.0) if tiny > 1e-10 else 0.0)
    got["dv_bound"] = u * got["dv"].abs() + tiny + fold(p_off.transpose(2, 3) @ do.abs()) + 1e-12
    return got
