"""The gradient of attention against its formula in binary64
(block_util.attention derives the bounds) and against differences of the
forward."""
import pytest

torch = pytest.importorskip("torch")

import block_util as B  # noqa: E402
from test_gpu_attention import TYPES, _i32, make  # noqa: E402
from video_vae_decoder_qkv_gb300 import attention, attention_backward, block  # noqa: E402

pytestmark = pytest.mark.gpu


def check(q, k, v, slopes=None, softcap=0.0, scale=None, dout=None, **masks):
    lens = {n: _i32(x) if not isinstance(x, bool) else x for n, x in masks.items()}
    kw = dict(softcap=softcap, slopes=slopes, scale=scale, **lens)
    if dout is None:
        g = torch.Generator(device="cuda").manual_seed(11)
        dout = torch.randn(q.shape, generator=g, device="cuda").to(q.dtype)
    out, lse = attention(q, k, v, **kw)
    grads = attention_backward(dout, q, k, v, out, lse, **kw)
    vis, dist = B.visible(q.shape[2], k.shape[2], q.shape[0], **masks)
    want = B.attention(q, k, v, vis, dist, dout=dout, softcap=softcap, slopes=slopes, scale=scale)
    assert block._fn("h3qk_attention_stuck")() == 0
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert got.dtype == q.dtype
        B.assert_within(got, want[name], want[name + "_bound"], name)
    assert (grads[0][~vis.any(2)[:, None].expand(q.shape[:3])] == 0).all()
    for t in grads[1:]:
        assert (t[~vis.any(1)[:, None].expand(t.shape[:3])] == 0).all()
    return out, lse, dout, grads


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("sq,sk", [(1, 1), (1, 200), (128, 128), (129, 257), (300, 100), (700, 701)])
def test_sizes(dtype, dim, sq, sk):
    check(*make(dtype, 1, 2, 2, sq, sk, dim))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (5, 1), (40, 8), (16, 1)])
@pytest.mark.parametrize("s", [60, 128, 333])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_heads(dtype, heads, kv_heads, s, causal):
    check(*make(dtype, 2, heads, kv_heads, s, s, 64), causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("s", [1, 90, 128, 300, 513])
def test_causal_and_prefix(dtype, dim, s):
    q, k, v = make(dtype, 2, 2, 1, s, s, dim)
    check(q, k, v, causal=True)
    check(q, k, v, causal=True, prefix_lens=[s // 3, s + 5])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sq,sk", [(7, 333), (150, 333), (333, 333)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("heads", [4, 2])
def test_lengths_that_leave_rows_empty(dtype, sq, sk, causal, heads):
    q, k, v = make(dtype, 4, heads, 2, sq, sk, 64, seed=2)
    check(q, k, v, causal=causal, kv_lens=[0, 333, 129, max(1, sk // 2)])
    check(q, k, v, causal=causal, q_lens=[0, sq, max(1, sq // 2), 1], kv_lens=[50, 333, 256, 1])
    check(q, k, v, causal=causal, kv_lens=[333, 0, 100, 7], q_starts=[-3, 5, 99, 6])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("offsets", [[0, 700], [0, 1, 2, 3, 700], [0, 0, 300, 300, 556, 640], [0, 0], [0, 256, 512],
                                     [0, 128, 700]])
def test_documents(dtype, dim, causal, offsets):
    q, k, v = make(dtype, 1, 3, 1, 700, 700, dim, seed=3)
    check(q, k, v, causal=causal, doc_offsets=offsets)
    if causal:
        check(q, k, v, causal=True, doc_offsets=offsets, prefix_lens=[7 * i for i in range(len(offsets) - 1)])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sq,sk", [(2, 40), (400, 400)])
def test_capped_scores_and_distance(dtype, dim, sq, sk):
    q, k, v = make(dtype, 2, 4, 2, sq, sk, dim, gain=2.5)
    slopes = torch.tensor([0.5, 0.1, 0.01, -0.02], device="cuda")
    check(q, k, v, softcap=20.0)
    check(q, k, v, softcap=5.0, causal=True)
    check(q, k, v, slopes=slopes)
    check(q, k, v, slopes=slopes, softcap=30.0, causal=True, kv_lens=[sk, sk // 2 + 1])
    check(q, k, v, scale=0.3)


@pytest.mark.parametrize("heads", [1, 5])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_long_rows_that_end_inside_a_tile(heads, dim, causal):
    """More query tiles than the ring holds, the last of each head partly past the rows that attend."""
    q, k, v = make(torch.bfloat16, 2, heads, 1, 1700, 1700, dim, seed=6)
    check(q, k, v, causal=causal, q_lens=[1650, 1409], kv_lens=[1700, 1409])
    q, k, v = q[:1], k[:1], v[:1]
    check(q, k, v, causal=causal, doc_offsets=[0, 1100, 1101, 1333, 1690])


def test_long_flat_rows_in_fp16():
    """Weights near 1/20,000, where an unscaled fp16 weight would be subnormal."""
    q, k, v = make(torch.float16, 1, 1, 1, 140, 20000, 64)
    check(q * 0.1, k, v)


@pytest.mark.parametrize("heads", [2, 4])
def test_rows_that_take_no_part_leave_no_mark(heads):
    """Unwritten query, key, value and gradient rows, with NaN and infinities."""
    q, k, v = make(torch.bfloat16, 2, heads, 2, 300, 300, 128)
    ql, kl = [210, 300], [170, 128]
    kw = dict(q_lens=_i32(ql), kv_lens=_i32(kl), causal=True)
    dout = torch.randn_like(q)
    out, lse = attention(q, k, v, **kw)
    want = attention_backward(dout, q, k, v, out, lse, **kw)
    for b in range(2):
        q[b, :, ql[b]:] = float("nan")
        dout[b, :, ql[b]:] = float("inf")
        k[b, :, kl[b]:] = float("-inf")
        v[b, :, kl[b]:] = float("nan")
    out2, lse2 = attention(q, k, v, **kw)
    got = attention_backward(dout, q, k, v, out2, lse2, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_documents_do_not_leak():
    q, k, v = make(torch.bfloat16, 1, 4, 2, 600, 600, 64)
    kw = dict(doc_offsets=_i32([0, 130, 200, 470]))
    dout = torch.randn_like(q)
    out, lse = attention(q, k, v, **kw)
    want = attention_backward(dout, q, k, v, out, lse, **kw)
    for t in (q, k, v, dout):
        t[:, :, 130:200] = float("nan")
        t[:, :, 470:] = float("inf")
    out, lse = attention(q, k, v, **kw)
    got = attention_backward(dout, q, k, v, out, lse, **kw)
    keep = [*range(130), *range(200, 600)]
    assert all(torch.equal(a[:, :, keep], b[:, :, keep]) for a, b in zip(got, want))


def test_layouts_same_bits_and_graph():
    b, h, hk, s, d = 2, 4, 2, 260, 64
    packed = torch.randn(b, s, (h + 2 * hk) * d + 8, device="cuda").to(torch.bfloat16)
    q = packed[..., :h * d].unflatten(2, (h, d)).transpose(1, 2)
    k = packed[..., h * d:(h + hk) * d].unflatten(2, (hk, d)).transpose(1, 2)
    v = packed[..., (h + hk) * d:(h + 2 * hk) * d].unflatten(2, (hk, d)).transpose(1, 2)
    out, lse, dout, grads = check(q, k, v, causal=True)
    plain = attention_backward(dout.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), out.contiguous(), lse,
                               causal=True)
    assert all(torch.equal(x, y) for x, y in zip(grads, plain))
    mine = tuple(torch.full((b, s, n, d + 8), 3.0, device="cuda", dtype=q.dtype) for n in (h, hk, hk))
    views = [t[..., :d].transpose(1, 2) for t in mine]
    ws = torch.empty(b * h * s, device="cuda")
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        attention_backward(dout, q, k, v, out, lse, causal=True, grad_q=views[0], grad_k=views[1], grad_v=views[2],
                           workspace=ws, stream=side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(views, plain))
    assert all((t[..., d:] == 3).all() for t in mine)


def test_no_rows_or_no_keys():
    q, k, v = make(torch.float16, 2, 2, 2, 0, 140, 64)
    out, lse = attention(q, k, v)
    dq, dk, dv = attention_backward(q, q, k, v, out, lse)
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    q, k, v = make(torch.float16, 2, 2, 2, 140, 0, 64)
    out, lse = attention(q, k, v)
    dq, dk, dv = attention_backward(torch.ones_like(q), q, k, v, out, lse)
    assert (dq == 0).all() and dk.shape == dv.shape == k.shape


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("softcap", [0.0, 3.0])
def test_gradient_against_differences_of_the_forward(which, softcap):
    """sum(dout . out) along the gradient's direction.  Each of the n outputs (size s ~ 0.2) is rounded to 11 bits and
    its weights too: noise of about 2^-10 s sqrt(n) in the sum.  The step changes the sum by 300 times that; the slope
    then agrees to 3 % (rounding) plus the curvature, of second order in a step that moves the inputs by a few
    percent."""
    q, k, v = make(torch.float16, 1, 4, 2, 96, 96, 64, seed=5)
    v[..., 0] /= 10
    dout = torch.randn_like(q)
    kw = dict(causal=True, softcap=softcap)
    out, lse = attention(q, k, v, **kw)
    grad = attention_backward(dout, q, k, v, out, lse, **kw)[which].double()
    noise = 2 ** -10 * float(out.double().norm())
    step = 300 * noise / float(grad.norm()) * grad / grad.norm()
    at = [q, k, v]
    plus, minus = list(at), list(at)
    plus[which] = (at[which].double() + step / 2).half()
    minus[which] = (at[which].double() - step / 2).half()
    f = lambda t: float((dout.double() * attention(*t, **kw)[0].double()).sum())  # noqa: E731
    want = float((grad * (plus[which].double() - minus[which].double())).sum())
    assert abs((f(plus) - f(minus)) - want) <= 0.03 * abs(want)


@pytest.mark.parametrize("dim", [64, 128])
def test_unseen_rows_leave_no_mark_on_capped_scores(dim):
    """Unwritten rows that follow 1, 2 and 3 past a multiple of 4, and documents that end there."""
    q, k, v = make(torch.bfloat16, 3, 4, 2, 300, 300, dim)
    ql, kl = [211, 300, 130], [171, 129, 130]
    kw = dict(q_lens=_i32(ql), kv_lens=_i32(kl), softcap=20.0)
    dout = torch.randn_like(q)
    out, lse = attention(q, k, v, **kw)
    want = attention_backward(dout, q, k, v, out, lse, **kw)
    for b in range(3):
        q[b, :, ql[b]:] = float("nan")
        dout[b, :, ql[b]:] = float("inf")
        k[b, :, kl[b]:] = float("nan")
        v[b, :, kl[b]:] = float("nan")
    out2, lse2 = attention(q, k, v, **kw)
    got = attention_backward(dout, q, k, v, out2, lse2, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 8.0])
@pytest.mark.parametrize("cut", [1, 200, 333])
def test_keys_in_two_calls_joined_by_lse(dtype, dim, softcap, cut):
    """The keys in two parts: out and lse joined, and each part's backward from the joined ones.  The joined out is
    off by its own rounding, and by that of the parts and of their weights (each at most u sum p |v|): what
    out_bound holds.  Each part's dq is rounded once."""
    q, k, v = make(dtype, 2, 4, 2, 150, 400, dim, seed=12)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(13), device="cuda").to(dtype)
    parts = [(k[:, :, a:b], v[:, :, a:b]) for a, b in ((0, cut), (cut, 400))]
    (o1, l1), (o2, l2) = (attention(q, *p, softcap=softcap) for p in parts)
    lse = torch.logaddexp(l1, l2)
    out = ((l1 - lse).exp()[..., None] * o1.float() + (l2 - lse).exp()[..., None] * o2.float()).to(dtype)
    (q1, k1, v1), (q2, k2, v2) = (attention_backward(dout, q, *p, out, lse, softcap=softcap) for p in parts)
    vis, dist = B.visible(150, 400, 2)
    want = B.attention(q, k, v, vis, dist, dout=dout, softcap=softcap)
    B.assert_within(q1.double() + q2.double(), want["dq"],
                    want["dq_bound"] + B.U[dtype] * (q1.double().abs() + q2.double().abs()) + 2 * B.TINY[dtype], "dq")
    B.assert_within(torch.cat([k1, k2], 2), want["dk"], want["dk_bound"], "dk")
    B.assert_within(torch.cat([v1, v2], 2), want["dv"], want["dv_bound"], "dv")


def test_out_and_lse_of_more_keys_than_the_call_has():
    """Keys that hold all but a little of the weight elsewhere: delta is that of the given out."""
    q, k, v = make(torch.float16, 1, 2, 2, 200, 300, 64, seed=14)
    v[:, :, 150:] += 3  # the other part's values lean one way
    dout = torch.randn_like(q)
    out, lse = attention(q, k, v)
    _, dk, dv = attention_backward(dout, q, k[:, :, :150], v[:, :, :150], out, lse)
    vis, dist = B.visible(200, 300, 1)
    want = B.attention(q, k, v, vis, dist, dout=dout)
    B.assert_within(dk, want["dk"][:, :, :150], want["dk_bound"][:, :, :150], "dk")
    B.assert_within(dv, want["dv"][:, :, :150], want["dv_bound"][:, :, :150], "dv")


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 1, 150, 64), (2, 4, 1, 64), (1, 4, 150, 1)])
def test_an_expanded_gradient(shape):
    """What the sum of the output gives, or of some of its dimensions."""
    q, k, v = make(torch.bfloat16, 2, 4, 2, 150, 150, 64)
    out, lse = attention(q, k, v)
    dout = torch.randn(shape, device="cuda").to(q.dtype).expand(q.shape)
    want = attention_backward(dout.contiguous(), q, k, v, out, lse)
    assert all(torch.equal(a, b) for a, b in zip(attention_backward(dout, q, k, v, out, lse), want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("softcap,gain", [(1025.0, 1.0), (1025.0, 6.0), (3e4, 1.0), (1e6, 1.0), (1e30, 1.0)])
def test_large_caps(dtype, dim, softcap, gain):
    """A cap far above the scores: the gradients' bounds without the cap's share."""
    q, k, v = make(dtype, 1, 2, 1, 300, 300, dim, seed=15, gain=gain)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(17), device="cuda").to(dtype)
    vis, dist = B.visible(300, 300, 1, causal=True)
    for slopes in (None, torch.tensor([0.02, 0.0], device="cuda")):
        kw = dict(softcap=softcap, slopes=slopes, causal=True)
        out, lse = attention(q, k, v, **kw)
        grads = attention_backward(dout, q, k, v, out, lse, **kw)
        want = B.attention(q, k, v, vis, dist, dout=dout, softcap=softcap, slopes=slopes)
        bound = B.attention(q, k, v, vis, dist, dout=dout, slopes=slopes)
        for name, got in zip(("dq", "dk", "dv"), grads):
            B.assert_within(got, want[name], bound[name + "_bound"], name)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_keys_past_the_last_row_get_zeros_whatever_they_hold(softcap, bad):
    """Causal rows that end before the keys do, and items whose rows all come before the first key."""
    q, k, v = make(torch.float16, 4, 4, 2, 70, 300, 64, seed=18)
    starts = [20, 229, 240, -80]
    for b, start in enumerate(starts):
        k[b, :, max(start + 70, 0):] = bad
        v[b, :, max(start + 70, 0):] = bad
    check(q, k, v, causal=True, q_starts=starts, softcap=softcap)
    check(q, k, v, causal=True, q_starts=starts, softcap=softcap, kv_lens=[299, 256, 300, 300])
