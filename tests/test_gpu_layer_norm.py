"""Layer norm and its gradient against their formulas in binary64.

Bounds: a sum of n binary32 terms in the kernels has at most 32 sequential
additions a thread and 10 levels of pairs above it, so its error is below
48 u sum|terms| (u = 2^-24); the weight gradients add at most all rows in
sequence.  With k = max(1, mean|x| rstd) the error of xh = (x - mean) rstd is
then below 64 u (k + |xh|).  Each result is rounded once to its type."""
import pytest

torch = pytest.importorskip("torch")

import block_util as B  # noqa: E402
from video_vae_decoder_qkv_gb300 import layer_norm, layer_norm_backward  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _make(dtype, rows, width, batch=1, affine="shared", offset=0.5, pad=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, width + pad, generator=g, device="cuda")
    x[:, :max(1, width // 100)] *= 20
    x = (x + offset).to(dtype)[:, :width]
    dy = torch.randn(rows, width + pad, generator=g, device="cuda").to(dtype)[:, :width]
    w = b = None
    if affine != "none":
        shape = (width,) if affine == "shared" else (batch, width)
        w = 1 + 0.3 * torch.randn(shape, generator=g, device="cuda")
        b = 0.2 * torch.randn(shape, generator=g, device="cuda")
    return x, dy, w, b


def _check(x, dy, w, b, batch, **kw):
    dtype, (rows, width) = x.dtype, x.shape
    y, stats = layer_norm(x, w, b, eps=EPS, batch=batch)
    dx, dw, db = layer_norm_backward(dy, x, w, stats, batch=batch, **kw)
    assert y.dtype == dx.dtype == dtype
    want, mean, rstd = B.layer_norm(x, w, b, EPS, batch)
    k = (x.double().abs().mean(1) * rstd).clamp(min=1.0)[:, None]
    xh = (x.double() - mean[:, None]) * rstd[:, None]
    xh_off = 64 * B.U32 * (k + xh.abs())
    wide = torch.ones(1, 1, dtype=torch.float64, device="cuda") if w is None else \
        w.double().abs().reshape(-1, 1, width).expand(batch if w.dim() == 2 else 1, rows // (batch if w.dim() == 2 else 1), width).reshape(rows, width)
    B.assert_within(y, want, B.U[dtype] * want.abs() + B.TINY[dtype] + 2 * xh_off * wide + 4 * B.U32 * want.abs(), "y")
    B.assert_within(stats[:, 0], mean, 64 * B.U32 * x.double().abs().mean(1), "mean")
    B.assert_within(stats[:, 1], rstd, 128 * B.U32 * k[:, 0] * rstd, "rstd")
    want_dx, want_dw, want_db = B.layer_norm_backward(dy, x, w, EPS, batch)
    g = dy.double().abs() * wide
    size = rstd[:, None] * (g + g.mean(1, keepdim=True) + xh.abs() * (g * xh.abs()).mean(1, keepdim=True))
    # xh enters the last term twice, and its error (relative to k) with it
    off = 256 * B.U32 * k * (size + rstd[:, None] * g.mean(1, keepdim=True) * (1 + xh.abs()))
    B.assert_within(dx, want_dx, B.U[dtype] * want_dx.abs() + B.TINY[dtype] + off, "dx")
    if w is None:
        assert dw is None and db is None
        return
    per = lambda t: t if w.dim() == 2 else t.sum(0)  # noqa: E731
    d = dy.double().abs().reshape(batch, -1, width)
    depth = rows + 64
    B.assert_within(dw, per(want_dw).reshape(w.shape),
                    per((d * (depth * B.U32 * xh.abs() + 2 * xh_off).reshape(d.shape)).sum(1)).reshape(w.shape) + 1e-30, "dw")
    B.assert_within(db, per(want_db).reshape(w.shape), per((d * depth * B.U32).sum(1)).reshape(w.shape) + 1e-30, "db")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 8), (3, 64), (5, 127), (17, 250), (33, 256), (9, 512), (700, 1024),
                                        (40, 1026), (21, 1013), (12, 5120), (3, 8190), (5, 8191), (4, 16384), (2, 16382),
                                        (2, 16383)])
def test_sizes(dtype, rows, width):
    _check(*_make(dtype, rows, width), 1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("affine", ["shared", "batch", "none"])
@pytest.mark.parametrize("batch,per,width", [(3, 1, 96), (2, 333, 640), (4, 50, 1100)])
def test_weights_per_item(dtype, affine, batch, per, width):
    _check(*_make(dtype, batch * per, width, batch, affine, seed=batch), batch)


@pytest.mark.parametrize("pad", [1, 2, 4, 8, 24])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_strides_and_offsets(dtype, pad):
    x, dy, w, b = _make(dtype, 30, 640, pad=pad)
    _check(x, dy, w, b, 1)
    # rows that start one element into a buffer
    big = torch.zeros(30 * 640 + 1, dtype=dtype, device="cuda")
    big[1:] = x.reshape(-1)
    _check(big[1:].view(30, 640), dy, w[:], b, 1)


def test_weights_off_a_16_byte_boundary():
    x, dy, w, b = _make(torch.float16, 20, 512)
    w1, b1 = torch.zeros(513, device="cuda"), torch.zeros(513, device="cuda")
    w1[1:], b1[1:] = w, b
    _check(x, dy, w1[1:], b1[1:], 1)


def test_a_mean_far_above_the_deviation():
    """Where mean^2 exceeds the variance ten million times over, E[x^2] - mean^2 would hold no digit."""
    x, dy, w, b = _make(torch.float32, 20, 1000, offset=3000.0)
    _check(x, dy, w, b, 1)


def test_constant_rows_and_one_column():
    x = torch.full((4, 256), 3.0, device="cuda", dtype=torch.bfloat16)
    y, stats = layer_norm(x, eps=EPS)
    assert (y == 0).all()
    assert torch.allclose(stats[:, 1], torch.full((4,), 1000.0, device="cuda"), rtol=1e-6)
    dx, _, _ = layer_norm_backward(torch.ones_like(x), x, None, stats)
    assert (dx == 0).all()


def test_a_bad_row_stays_its_own():
    x, dy, w, b = _make(torch.float16, 24, 384)
    x = x.clone()
    x[5, 3], x[11, 380] = float("nan"), float("inf")
    y, stats = layer_norm(x, w, b, eps=EPS)
    dx, _, _ = layer_norm_backward(dy, x, w, stats)
    bad = torch.zeros(24, dtype=torch.bool, device="cuda")
    bad[5] = bad[11] = True
    for t in (y, dx):
        assert t[bad].isnan().all() and t[~bad].isfinite().all()


def test_no_rows_give_zero_weight_gradients():
    x = torch.empty(0, 320, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(320, device="cuda")
    y, stats = layer_norm(x, w, w)
    dx, dw, db = layer_norm_backward(x, x, w, stats)
    assert y.shape == dx.shape == (0, 320) and (dw == 0).all() and (db == 0).all()


def test_same_bits_every_time_and_without_weight_gradients():
    x, dy, w, b = _make(torch.bfloat16, 3000, 1024)
    _, stats = layer_norm(x, w, b)
    one, two = layer_norm_backward(dy, x, w, stats), layer_norm_backward(dy, x, w, stats)
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    dx, dw, db = layer_norm_backward(dy, x, w, stats, need_weight_grad=False)
    assert torch.equal(dx, one[0]) and dw is None and db is None


def test_caller_buffers_stream_and_graph():
    x, dy, w, b = _make(torch.float16, 100, 768)
    want_y, want_stats = layer_norm(x, w, b)
    want = layer_norm_backward(dy, x, w, want_stats)
    from video_vae_decoder_qkv_gb300 import block

    y, stats, dx = torch.empty_like(x), torch.empty_like(want_stats), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(block._size("h3qk_layer_norm_backward_workspace_bytes", x.device, 100, 768, 1), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer_norm(x, w, b, out=y, stats=stats, stream=side)
        layer_norm_backward(dy, x, w, stats, out=dx, grad_weight=dw, grad_bias=db, workspace=ws, stream=side)
    for _ in range(2):
        for t in (y, stats, dx, dw, db):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((y, stats, dx, dw, db), (want_y, want_stats, *want)):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("which", ["x", "weight", "bias"])
def test_gradient_against_differences(which):
    """sum(dy y) along the gradient's own direction, central differences in binary32.  With a step s the
    truncation is of order s^2 and the rounding u |L| / s: 1e-3 of the derivative at s = 1e-2 covers both."""
    x, dy, w, b = _make(torch.float32, 12, 200, seed=4)
    _, stats = layer_norm(x, w, b)
    dx, dw, db = layer_norm_backward(dy, x, w, stats)
    grad = {"x": dx, "weight": dw, "bias": db}[which]
    v = grad / grad.double().norm().float()
    f = lambda t: float((dy.double() * layer_norm(*t)[0].double()).sum())  # noqa: E731
    at = {"x": x, "weight": w, "bias": b}
    plus = f(tuple(at[n] + (1e-2 * v if n == which else 0) for n in at))
    minus = f(tuple(at[n] - (1e-2 * v if n == which else 0) for n in at))
    slope = float((grad.double() * v.double()).sum())
    assert abs((plus - minus) / 2e-2 - slope) <= 1e-3 * slope


_FIRST_CALLS = """
import sys
sys.path[:0] = sys.argv[1:]
import torch
import test_gpu_layer_norm as T
from video_vae_decoder_qkv_gb300 import layer_norm, layer_norm_backward
# Widths whose rows ahead take 48 KiB of shared memory or just under it, beside what the kernel holds
# itself; by kind of row (chunks of 16 bytes, pairs, single elements) and direction.
for dtype, forward, backward in ((torch.float16, (6000, 6110, 6127), (2880, 3050, 3047)),
                                 (torch.bfloat16, (6144, 6114, 6113), (2576, 3038, 3061)),
                                 (torch.float32, (2880, 3061), (2000, 2033))):
    for width in backward:
        x, dy, w, b = T._make(dtype, 9, width)
        _, mean, rstd = T.B.layer_norm(x, None, None, T.EPS, 1)
        layer_norm_backward(dy, x, w, torch.stack([mean, rstd], 1).float())
    for width in forward:
        x, dy, w, b = T._make(dtype, 9, width)
        layer_norm(x, w, b)
    for width in (*backward, *forward):
        T._check(*T._make(dtype, 9, width), 1)
"""


def test_widths_at_the_shared_memory_limit_as_first_calls():
    """A fresh process: a wider call would have raised a kernel's limit for good."""
    import os
    import subprocess
    import sys

    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS, here, os.path.dirname(here)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("shape", [(1, 1), (1, 640), (30, 1)])
def test_an_expanded_gradient(shape):
    """What the sum of the output gives, or of its rows or columns."""
    x, _, w, b = _make(torch.float16, 30, 640)
    _, stats = layer_norm(x, w, b)
    dy = torch.randn(shape, device="cuda").half().expand(30, 640)
    want = layer_norm_backward(dy.contiguous(), x, w, stats)
    assert all(torch.equal(p, q) for p, q in zip(layer_norm_backward(dy, x, w, stats), want))
