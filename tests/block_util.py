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
