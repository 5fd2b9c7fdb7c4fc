"""The gradient of ``prepare`` against its formula in binary64 and against
differences of the forward.

Bounds: the sums over D <= 256 channels have at most 8 sequential additions
and 5 levels of pairs, so with the products' roundings a result is off by at
most 32 u of the terms it is made of (u = 2^-24; |sin|, |cos| are found to
2^-22), then rounded once to its type; a weight gradient adds at most
rows * heads terms in sequence."""
import pytest

torch = pytest.importorskip("torch")

import block_util as B  # noqa: E402
from video_vae_decoder_qkv_gb300 import prepare, prepare_backward  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _make(dtype, batch, seq, heads, dim, n_axes, pad=0, seed=0, layout="head_major"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(batch * seq, 3 * heads * dim + pad, generator=g, device="cuda").to(dtype)
    wq = 0.5 + torch.rand(dim, generator=g, device="cuda")
    wk = 0.5 + torch.rand(dim, generator=g, device="cuda")
    pos = torch.randint(0, 70, (batch * seq, n_axes), generator=g, device="cuda", dtype=torch.int32)
    shape = (batch, heads, seq, dim) if layout == "head_major" else (batch, seq, heads, dim)
    grads = tuple(torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(3))
    return qkv, wq, wk, pos, grads


def _want(qkv, wq, wk, pos, grads, heads, dim, rotary, axis_dims, batch, valid, layout="head_major"):
    """(dqkv, dwq, dwk) in binary64 and the sizes of the terms behind each."""
    tokens = qkv.shape[0]
    seq = tokens // batch
    ang = B.angles(pos, rotary, axis_dims)
    valid = torch.as_tensor(valid, device="cuda").reshape(-1, 1)
    keep = (torch.arange(seq, device="cuda")[None] < valid).expand(batch, seq).reshape(-1, 1, 1)
    x = qkv[:, :3 * heads * dim].reshape(tokens, 3, heads, dim).double()
    out, size, dws, dw_size = torch.zeros_like(x), torch.zeros_like(x), [], []
    for t, w in ((0, wq), (1, wk), (2, None)):
        dy = grads[t].double()
        dy = (dy.transpose(1, 2) if layout == "head_major" else dy).reshape(tokens, heads, dim)
        dy = torch.where(keep, dy, 0.0)
        if w is None:
            out[:, t] = dy
            continue
        xt = torch.where(keep, x[:, t], 0.0)
        inv = ((xt * xt).mean(2, keepdim=True) + EPS) ** -0.5
        dn, dn_size = dy.clone(), dy.abs()
        if rotary:
            z = torch.view_as_complex(dy[..., :rotary].reshape(tokens, heads, rotary // 2, 2).contiguous())
            z = z * torch.polar(torch.ones_like(ang), -ang)[:, None, :]
            dn = torch.cat([torch.view_as_real(z).reshape(tokens, heads, rotary), dy[..., rotary:]], 2)
            r = dy[..., :rotary].reshape(tokens, heads, rotary // 2, 2).abs().sum(3, keepdim=True)
            dn_size = torch.cat([r.expand(-1, -1, -1, 2).reshape(tokens, heads, rotary), dy[..., rotary:].abs()], 2)
        g = dn * w.double()
        out[:, t] = inv * g - xt * inv ** 3 * (g * xt).mean(2, keepdim=True)
        gs = dn_size * w.double().abs()
        size[:, t] = inv * gs + xt.abs() * inv ** 3 * (gs * xt.abs()).mean(2, keepdim=True)
        dws.append((dn * xt * inv).sum((0, 1)))
        dw_size.append((dn_size * xt.abs() * inv).sum((0, 1)))
    return out.reshape(tokens, -1), size.reshape(tokens, -1), dws, dw_size


def _check(dtype, batch, seq, heads, dim, rotary, n_axes=3, valid=None, pad=0, layout="head_major", valid_lens=None,
           axis_dims=None, seed=0):
    qkv, wq, wk, pos, grads = _make(dtype, batch, seq, heads, dim, n_axes, pad, seed, layout)
    axis_dims = axis_dims or (rotary // n_axes,) * n_axes
    keep = seq if valid is None else valid
    vl = None if valid_lens is None else torch.tensor(valid_lens, dtype=torch.int32, device="cuda")
    got, gq, gk = prepare_backward(*grads, qkv, wq, wk, pos, heads=heads, head_dim=dim, rotary_dim=rotary, batch=batch,
                                   valid_len=valid, n_axes=n_axes, axis_dims=axis_dims, eps=EPS, layout=layout,
                                   valid_lens=vl)
    want, size, dws, dw_size = _want(qkv, wq, wk, pos, grads, heads, dim, rotary, axis_dims, batch,
                                     keep if valid_lens is None else valid_lens, layout)
    assert got.dtype == dtype
    B.assert_within(got, want, B.U[dtype] * want.abs() + B.TINY[dtype] + 32 * B.U32 * size, "grad_qkv")
    depth = batch * seq * heads + 64
    for name, g, w, s in (("grad_wq", gq, dws[0], dw_size[0]), ("grad_wk", gk, dws[1], dw_size[1])):
        B.assert_within(g, w, depth * B.U32 * s + 1e-30, name)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,rotary", [(1, 8, 6), (3, 16, 12), (2, 24, 24), (4, 64, 48), (5, 80, 60), (3, 128, 96),
                                              (2, 136, 96), (1, 256, 192), (3, 64, 0)])
@pytest.mark.parametrize("seq", [1, 7, 48])
def test_sizes(dtype, heads, dim, rotary, seq):
    _check(dtype, 1, seq, heads, dim, rotary)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_one_axis_uneven_axes_and_an_odd_rotary_width(dtype):
    _check(dtype, 1, 50, 3, 128, 128, n_axes=1)
    _check(dtype, 1, 50, 3, 128, 92, axis_dims=(28, 30, 34))
    _check(dtype, 1, 50, 2, 40, 26, n_axes=1)


@pytest.mark.parametrize("layout", ["head_major", "token_major"])
def test_valid_prefix_strides_and_layouts(layout):
    _check(torch.bfloat16, 2, 33, 4, 64, 48, valid=20, pad=16, layout=layout)
    _check(torch.float16, 3, 21, 2, 128, 96, layout=layout, valid_lens=[0, 21, 13])
    _check(torch.float16, 1, 9, 2, 64, 48, valid=0, layout=layout)


def test_rows_past_the_prefix_are_not_read():
    """Unwritten memory past the prefix, with infinities and NaN, leaves no mark."""
    qkv, wq, wk, pos, grads = _make(torch.bfloat16, 1, 40, 2, 64, 3)
    kw = dict(heads=2, head_dim=64, rotary_dim=48, valid_len=29)
    want = prepare_backward(*grads, qkv, wq, wk, pos, **kw)
    qkv[29:] = float("nan")
    for g in grads:
        g[:, :, 29:] = float("inf")
    got = prepare_backward(*grads, qkv, wq, wk, pos, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (got[0][29:] == 0).all()


def test_many_rows_many_heads_and_the_same_bits():
    _check(torch.bfloat16, 2, 2000, 16, 64, 48, valid=1990, seed=3)
    qkv, wq, wk, pos, grads = _make(torch.float16, 1, 3000, 7, 128, 3)
    kw = dict(heads=7, head_dim=128, rotary_dim=96)
    one, two = (prepare_backward(*grads, qkv, wq, wk, pos, **kw) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_no_rows():
    qkv, wq, wk, pos, grads = _make(torch.float16, 1, 0, 2, 64, 3)
    got, gq, gk = prepare_backward(*grads, qkv, wq, wk, pos, heads=2, head_dim=64, rotary_dim=48)
    assert got.shape == (0, 384) and (gq == 0).all() and (gk == 0).all()


def test_zero_rows_stay_finite():
    qkv, wq, wk, pos, grads = _make(torch.float16, 1, 16, 2, 64, 3)
    qkv.zero_()
    grads = tuple(g * 1e-3 for g in grads)
    got, gq, gk = prepare_backward(*grads, qkv, wq, wk, pos, heads=2, head_dim=64, rotary_dim=48)
    assert got.isfinite().all() and (gq == 0).all() and (gk == 0).all()


@pytest.mark.parametrize("which", ["qkv", "wq", "wk"])
def test_gradient_against_differences_of_the_forward(which):
    """sum(dy . (q, k, v)) of ``prepare`` itself along the gradient's direction.  The forward rounds each value
    twice to 11 bits; with n such values of size ~1 the sum's rounding is about 2^-11 sqrt(n) sqrt(2), which a step
    of norm s divides: the test takes a step whose change is 200 times that, and allows 3 %."""
    batch, seq, heads, dim = 1, 64, 4, 64
    qkv, wq, wk, pos, grads = _make(torch.float16, batch, seq, heads, dim, 3, seed=9)
    kw = dict(heads=heads, head_dim=dim, rotary_dim=48)
    dqkv, dwq, dwk = prepare_backward(*grads, qkv, wq, wk, pos, **kw)
    grad = {"qkv": dqkv, "wq": dwq, "wk": dwk}[which].double()
    n = 3 * seq * heads * dim
    noise = 2 ** -11 * (2 * n) ** 0.5
    at = {"qkv": qkv, "wq": wq, "wk": wk}
    step = 200 * noise / float(grad.norm()) * grad / grad.norm()
    plus, minus = dict(at), dict(at)
    plus[which] = (at[which].double() + step / 2).to(at[which].dtype)
    minus[which] = (at[which].double() - step / 2).to(at[which].dtype)

    def f(a):
        out = prepare(a["qkv"], a["wq"], a["wk"], pos, eps=EPS, **kw)[:3]
        return sum(float((d.double() * o.double()).sum()) for d, o in zip(grads, out))

    want = float((grad * (plus[which].double() - minus[which].double())).sum())
    assert abs((f(plus) - f(minus)) - want) <= 0.03 * abs(want)


@pytest.mark.parametrize("size,eps", [(1e13, 1e-6), (1e15, 1e-6), (1e17, 1e-6), (1.0, 0.0), (1e-14, 0.0), (1e-17, 0.0)])
def test_rows_of_any_size(monkeypatch, size, eps):
    """Rows whose inverse norm has a cube outside binary32's range."""
    import sys

    monkeypatch.setattr(sys.modules[__name__], "EPS", eps)
    qkv, wq, wk, pos, grads = _make(torch.bfloat16, 1, 48, 3, 64, 3)
    qkv = (qkv.double() * size).to(torch.bfloat16)
    got, gq, gk = prepare_backward(*grads, qkv, wq, wk, pos, heads=3, head_dim=64, rotary_dim=48, eps=eps)
    want, terms, dws, dw_terms = _want(qkv, wq, wk, pos, grads, 3, 64, 48, (16, 16, 16), 1, 48)
    dtype = torch.bfloat16
    B.assert_within(got, want, B.U[dtype] * want.abs() + B.TINY[dtype] + 32 * B.U32 * terms, "grad_qkv")
    for g, w, s in ((gq, dws[0], dw_terms[0]), (gk, dws[1], dw_terms[1])):
        B.assert_within(g, w, (48 * 3 + 64) * B.U32 * s + 1e-30, "grad_w")


def test_expanded_gradients():
    """What the sum of an output gives."""
    qkv, wq, wk, pos, grads = _make(torch.float16, 2, 21, 3, 64, 3)
    kw = dict(heads=3, head_dim=64, rotary_dim=48, batch=2)
    grads = [g[:1, :1, :1, :1].expand(g.shape) for g in grads]
    want = prepare_backward(*(g.contiguous() for g in grads), qkv, wq, wk, pos, **kw)
    assert all(torch.equal(a, b) for a, b in zip(prepare_backward(*grads, qkv, wq, wk, pos, **kw), want))
