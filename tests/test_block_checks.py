"""Refusals of the attention block's operators, without a GPU: the binding on
meta tensors, and the C-ABI on fake addresses that every call rejects before
it would touch them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from video_vae_decoder_qkv_gb300 import (attention, attention_backward, block, h3qk, layer_norm,  # noqa: E402
                                         layer_norm_backward, prepare_backward)

M = torch.device("meta")
F16, F32, I32 = torch.float16, torch.float32, torch.int32
A = 0x10000000


def t(*shape, dtype=F16):
    return torch.empty(shape, dtype=dtype, device=M)


@pytest.fixture
def no_gpu():
    """Fake addresses must never reach a kernel: only where no GPU exists."""
    if torch.cuda.is_available():
        pytest.skip("fake-address checks run only on hosts without a GPU")


@pytest.mark.parametrize("args,kw,error", [
    ((t(4, 8, dtype=torch.float64),), {}, TypeError),
    ((t(4, 8, 2),), {}, ValueError),
    ((t(8, 4).t(),), {}, ValueError),
    ((t(1, 8).expand(4, 8),), {}, ValueError),
    ((t(5, 8),), dict(batch=2), ValueError),
    ((t(4, 8), t(8)), {}, TypeError),
    ((t(4, 8), t(7, dtype=F32)), {}, ValueError),
    ((t(4, 8), t(3, 8, dtype=F32)), dict(batch=2), ValueError),
    ((t(4, 8), t(8, dtype=F32), t(2, 8, dtype=F32)), dict(batch=2), ValueError),
    ((t(4, 8), t(16, dtype=F32)[::2]), {}, ValueError),
    ((t(4, 8),), dict(out=t(4, 7)), ValueError),
    ((t(4, 8),), dict(out=t(4, 8, dtype=F32)), TypeError),
    ((t(4, 8),), dict(stats=t(4, dtype=F32)), ValueError),
])
def test_layer_norm_refuses(args, kw, error):
    with pytest.raises(error):
        layer_norm(*args, **kw)


@pytest.mark.parametrize("dy,x,w,stats,kw,error", [
    (t(4, 8, dtype=F32), t(4, 8), None, t(4, 2, dtype=F32), {}, TypeError),
    (t(4, 7), t(4, 8), None, t(4, 2, dtype=F32), {}, ValueError),
    (t(4, 8), t(4, 8), None, t(3, 2, dtype=F32), {}, ValueError),
    (t(4, 8), t(4, 8), None, None, {}, ValueError),
    (t(4, 8), t(4, 8), t(9, dtype=F32), t(4, 2, dtype=F32), {}, ValueError),
    (t(4, 8), t(4, 8), None, t(4, 2, dtype=F32), dict(out=t(2, 8)), ValueError),
])
def test_layer_norm_backward_refuses(dy, x, w, stats, kw, error):
    with pytest.raises(error):
        layer_norm_backward(dy, x, w, stats, **kw)


def _prep(**kw):
    a = dict(gq=t(1, 4, 32, 64), gk=t(1, 4, 32, 64), gv=t(1, 4, 32, 64), qkv=t(32, 768), wq=t(64, dtype=F32),
             wk=t(64, dtype=F32), pos=t(32, 3, dtype=I32))
    more = {k: v for k, v in kw.items() if k not in a}
    a.update({k: v for k, v in kw.items() if k in a})
    return prepare_backward(*a.values(), heads=4, head_dim=64, rotary_dim=48, **more)


@pytest.mark.parametrize("kw,error", [
    (dict(qkv=t(32, 768, dtype=F32)), TypeError), (dict(qkv=t(32, 760)), ValueError),
    (dict(gq=t(1, 4, 31, 64)), ValueError), (dict(gk=t(1, 4, 32, 64, dtype=torch.bfloat16)), TypeError),
    (dict(gv=t(1, 4, 64, 32).transpose(2, 3)), ValueError), (dict(wq=t(32, dtype=F32)), ValueError),
    (dict(pos=t(31, 3, dtype=I32)), ValueError), (dict(batch=3), ValueError), (dict(out=t(32, 767)), ValueError),
    (dict(grad_wq=t(63, dtype=F32)), ValueError), (dict(layout="other"), KeyError),
    (dict(valid_lens=t(2, dtype=I32)), ValueError),
])
def test_prepare_backward_refuses(kw, error):
    with pytest.raises(error):
        _prep(**kw)


@pytest.mark.parametrize("q,k,v,kw,error", [
    (t(1, 4, 9, 64, dtype=F32), t(1, 4, 9, 64), t(1, 4, 9, 64), {}, TypeError),
    (t(4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), {}, ValueError),
    (t(1, 4, 9, 64), t(1, 3, 9, 64), t(1, 3, 9, 64), {}, ValueError),
    (t(1, 4, 9, 64), t(1, 0, 9, 64), t(1, 0, 9, 64), {}, ValueError),
    (t(1, 4, 9, 64), t(2, 4, 9, 64), t(2, 4, 9, 64), {}, ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 72), t(1, 4, 9, 72), {}, ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64, dtype=torch.bfloat16), t(1, 4, 9, 64), {}, TypeError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 8, 64), {}, ValueError),
    (t(1, 4, 64, 9).transpose(2, 3), t(1, 4, 9, 64), t(1, 4, 9, 64), {}, ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(out=t(1, 4, 9, 32)), ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(lse=t(1, 4, 8, dtype=F32)), ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(slopes=t(3, dtype=F32)), ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(kv_lens=t(2, dtype=I32)), ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(q_lens=t(1, dtype=torch.int64)), TypeError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(doc_offsets=t(1, dtype=I32)), ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(doc_offsets=t(3, dtype=I32), kv_lens=t(1, dtype=I32)), ValueError),
    (t(1, 4, 9, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(doc_offsets=t(3, dtype=I32), prefix_lens=t(3, dtype=I32)), ValueError),
    (t(2, 4, 9, 64), t(2, 4, 9, 64), t(2, 4, 9, 64), dict(doc_offsets=t(3, dtype=I32)), ValueError),
    (t(1, 4, 8, 64), t(1, 4, 9, 64), t(1, 4, 9, 64), dict(doc_offsets=t(3, dtype=I32)), ValueError),
])
def test_attention_refuses(q, k, v, kw, error):
    with pytest.raises(error):
        attention(q, k, v, **kw)


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan")])
def test_attention_refuses_a_scale_that_is_not_positive(scale):
    q = t(1, 4, 9, 64)
    with pytest.raises(ValueError, match="scale"):
        attention(q, q, q, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        attention_backward(q, q, q, q, q, t(1, 4, 9, dtype=F32), scale=scale)


def test_operators_refuse_host_tensors():
    """The library would read host addresses on the device."""
    x, w = torch.ones(4, 8), torch.ones(8)
    q = torch.zeros(1, 2, 100, 64, dtype=F16)
    for call in (lambda: layer_norm(x, w), lambda: layer_norm_backward(x, x, None, torch.ones(4, 2)),
                 lambda: attention(q, q, q)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()


@pytest.mark.parametrize("name,bad,error", [
    ("grad_out", t(1, 4, 9, 64, dtype=F32), TypeError), ("grad_out", t(1, 4, 8, 64), ValueError),
    ("out", t(1, 4, 9, 32), ValueError), ("lse", t(1, 4, 8, dtype=F32), ValueError), ("lse", None, ValueError),
    ("grad_q", t(1, 4, 9, 32), ValueError), ("grad_k", t(1, 2, 8, 64), ValueError),
    ("grad_v", t(1, 2, 9, 64, dtype=F32), TypeError),
])
def test_attention_backward_refuses(name, bad, error):
    a = dict(grad_out=t(1, 4, 9, 64), q=t(1, 4, 9, 64), k=t(1, 2, 9, 64), v=t(1, 2, 9, 64), out=t(1, 4, 9, 64),
             lse=t(1, 4, 9, dtype=F32))
    a[name] = bad
    with pytest.raises(error):
        attention_backward(**a)


# --- the C-ABI ---------------------------------------------------------------

def _attn(backward=False, **kw):
    B, H, HK, S, D = 2, 4, 2, 300, 64
    f = dict(dtype=h3qk.FP16, batch=B, heads=H, kv_heads=HK, head_dim=D, causal=0, docs=0, reserved=0, scale=0.0,
             softcap=0.0, q_rows=S, kv_rows=S, q=A, k=A + 0x1000000, v=A + 0x2000000, out=A + 0x3000000,
             lse=A + 0x4000000, grad_out=A + 0x5000000, grad_q=A + 0x6000000, grad_k=A + 0x7000000,
             grad_v=A + 0x8000000, slopes=0, prefix_lens=0, doc_offsets=0, q_lens=0, kv_lens=0, q_starts=0,
             workspace=A + 0x9000000, workspace_bytes=1 << 24)
    row, key = (H * S * D, S * D, D), (HK * S * D, S * D, D)
    st = dict(q=row, k=key, v=key, out=row, grad_out=row, grad_q=row, grad_k=key, grad_v=key)
    for n in list(kw):
        if n.endswith("_strides"):
            st[n[:-8]] = kw.pop(n)
    f.update(kw)
    packed = block._ATTN.pack(*f.values(), *(x for s in st.values() for x in s))
    return block._fn("h3qk_attention_backward" if backward else "h3qk_attention")(packed, None)


INVALID, MISALIGNED, ALIAS = h3qk.ERR_INVALID_ARG, h3qk.ERR_MISALIGNED, h3qk.ERR_ALIAS
BOTH = [
    (dict(dtype=h3qk.E4M3), INVALID), (dict(dtype=block.FP32), INVALID), (dict(batch=0), INVALID),
    (dict(heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=136), INVALID),
    (dict(head_dim=60), INVALID), (dict(head_dim=0), INVALID), (dict(causal=2), INVALID), (dict(docs=-1), INVALID),
    (dict(reserved=1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("inf")), INVALID), (dict(q_rows=-1), INVALID),
    (dict(kv_rows=1 << 30), INVALID), (dict(docs=2, batch=1), INVALID), (dict(docs=2, doc_offsets=A - 64), INVALID),
    (dict(doc_offsets=A - 64), INVALID), (dict(prefix_lens=A - 64), INVALID), (dict(q=0), INVALID), (dict(v=0), INVALID),
    (dict(out=0), INVALID), (dict(lse=0), INVALID), (dict(q_strides=(76800, 19200, 56)), INVALID),
    (dict(k_strides=(0, 19200, 64)), INVALID), (dict(v_strides=(-38400, 19200, 64)), INVALID),
    (dict(q_strides=(1 << 40, 19200, 64)), INVALID), (dict(q=A + 8), MISALIGNED), (dict(k_strides=(38400, 19200, 68)), MISALIGNED),
    (dict(v_strides=(38404, 19200, 64)), MISALIGNED), (dict(lse=A + 0x4000002), MISALIGNED),
    (dict(slopes=A - 62), MISALIGNED), (dict(kv_lens=A - 62), MISALIGNED),
]


@pytest.mark.parametrize("kw,want", BOTH)
@pytest.mark.parametrize("backward", [False, True])
def test_attention_checks(no_gpu, backward, kw, want):
    assert _attn(backward, **kw) == want


@pytest.mark.parametrize("backward,kw,want", [
    (False, dict(out=A), ALIAS), (False, dict(out=A + 0x1000000 + 64), ALIAS), (False, dict(lse=A + 0x3000000), ALIAS),
    (False, dict(kv_lens=A + 0x4000000), ALIAS), (False, dict(out_strides=(76800, 64, 64)), ALIAS),
    (False, dict(q_rows=1, workspace=0), INVALID), (False, dict(q_rows=1, workspace_bytes=16), INVALID),
    (False, dict(q_rows=1, workspace=A + 0x9000008), MISALIGNED), (False, dict(q_rows=1, workspace=A + 0x3000000), ALIAS),
    (True, dict(grad_out=0), INVALID), (True, dict(grad_k=0), INVALID), (True, dict(workspace=0), INVALID),
    (True, dict(workspace_bytes=9599), INVALID), (True, dict(workspace=A + 0x9000004), MISALIGNED),
    (True, dict(grad_q=A + 0x5000000), ALIAS), (True, dict(grad_v=A + 0x7000000), ALIAS),
    (True, dict(grad_k=A + 0x4000000), ALIAS), (True, dict(workspace=A + 0x3000000), ALIAS),
    (True, dict(grad_k_strides=(38400, 64, 64)), ALIAS), (True, dict(grad_q=A + 0x6000008), MISALIGNED),
])
def test_attention_workspaces_and_aliases(no_gpu, backward, kw, want):
    assert _attn(backward, **kw) == want


def test_attention_null_call(no_gpu):
    assert block._fn("h3qk_attention")(None, None) == INVALID
    assert block._fn("h3qk_attention_backward")(None, None) == INVALID
    assert block._fn("h3qk_attention_workspace_bytes")(None) == 0


@pytest.mark.parametrize("backward", [False, True])
def test_a_valid_call_without_a_device_reports_cuda_error(no_gpu, backward):
    assert _attn(backward) == h3qk.ERR_CUDA
    assert h3qk.lib().h3qk_last_cuda_error() != 0
    assert _attn(backward, batch=1, docs=1, doc_offsets=A - 64) == h3qk.ERR_CUDA
    assert _attn(backward, q_rows=0, kv_rows=0) == h3qk.OK


def _ln(**kw):
    a = dict(x=A, dtype=h3qk.FP16, rows=10, width=64, stride=0, w=A + 0x100000, b=A + 0x101000, groups=1, eps=1e-6,
             out=A + 0x200000, stats=A + 0x300000)
    a.update(kw)
    return block._fn("h3qk_layer_norm")(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=h3qk.E4M3), INVALID), (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(width=16385), INVALID),
    (dict(groups=3), INVALID), (dict(groups=0), INVALID), (dict(stride=63), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(stats=0), INVALID),
    (dict(x=A + 1), MISALIGNED), (dict(stats=A + 0x300004), MISALIGNED), (dict(w=A + 0x100002), MISALIGNED),
    (dict(out=A + 64), ALIAS), (dict(stats=A + 0x200000), ALIAS), (dict(stats=A + 0x100000), ALIAS),
    (dict(), h3qk.ERR_CUDA), (dict(rows=0, x=0, out=0, stats=0), h3qk.OK),
])
def test_layer_norm_checks(no_gpu, kw, want):
    assert _ln(**kw) == want


def _ln_back(**kw):
    a = dict(dy=A + 0x400000, dy_stride=0, x=A, dtype=h3qk.FP16, rows=10, width=64, stride=0, w=A + 0x100000, groups=1,
             stats=A + 0x300000, dx=A + 0x500000, dw=A + 0x600000, db=A + 0x601000, ws=A + 0x700000, ws_bytes=1 << 24)
    a.update(kw)
    return block._fn("h3qk_layer_norm_backward")(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=0), INVALID), (dict(dy_stride=32), INVALID), (dict(stats=0), INVALID), (dict(dx=0), INVALID),
    (dict(ws=0), INVALID), (dict(ws_bytes=64), INVALID), (dict(ws=A + 0x700008), MISALIGNED),
    (dict(dw=A + 0x600002), MISALIGNED), (dict(dx=A + 0x400000), ALIAS), (dict(dw=A + 0x601000), ALIAS),
    (dict(ws=A + 0x300000), ALIAS), (dict(dx=A + 0x300000), ALIAS), (dict(), h3qk.ERR_CUDA),
    (dict(dw=0, db=0, ws=0, ws_bytes=0), h3qk.ERR_CUDA),
])
def test_layer_norm_backward_checks(no_gpu, kw, want):
    assert _ln_back(**kw) == want


def _prep_back(**kw):
    o = h3qk.default_opts()
    o.in_dtype = h3qk.BF16
    a = dict(gq=A + 0x1000000, gk=A + 0x2000000, gv=A + 0x3000000, qkv=A, wq=A + 0x500000, wk=A + 0x501000,
             pos=A + 0x502000, tokens=48, heads=4, dim=64, rotary=48, valid=48, out=A + 0x4000000, dwq=A + 0x600000,
             dwk=A + 0x601000, ws=A + 0x700000, ws_bytes=1 << 24)
    a.update(kw)
    return block._fn("h3qk_prepare_backward")(*a.values(), ctypes.byref(o), None)


@pytest.mark.parametrize("kw,want", [
    (dict(gq=0), INVALID), (dict(gv=0), INVALID), (dict(out=0), INVALID), (dict(qkv=0), INVALID), (dict(pos=0), INVALID),
    (dict(dim=60), INVALID), (dict(rotary=50), INVALID), (dict(valid=49), INVALID), (dict(ws=0), INVALID),
    (dict(ws_bytes=100), INVALID), (dict(gk=A + 0x2000008), MISALIGNED), (dict(out=A + 0x4000004), MISALIGNED),
    (dict(ws=A + 0x700004), MISALIGNED), (dict(dwq=A + 0x600002), MISALIGNED), (dict(out=A), ALIAS),
    (dict(out=A + 0x1000000), ALIAS), (dict(dwq=A + 0x601000), ALIAS), (dict(ws=A + 0x4000000), ALIAS),
    (dict(dwk=A + 0x500000), ALIAS), (dict(), h3qk.ERR_CUDA), (dict(dwq=0, dwk=0), h3qk.ERR_CUDA),
])
def test_prepare_backward_checks(no_gpu, kw, want):
    assert _prep_back(**kw) == want


def test_workspace_sizes():
    f = block._fn("h3qk_layer_norm_backward_workspace_bytes")
    assert 0 < f(10, 64, 1) <= f(1000, 64, 1) and f(10, 64, 3) == 0 and f(10, 0, 1) == 0 and f(-1, 64, 1) == 0
    f = block._fn("h3qk_prepare_backward_workspace_bytes")
    assert 0 < f(64) < f(128) and f(60) == 0 and f(512) == 0


@pytest.mark.parametrize("q_rows,kv_rows", [(4896, 4896), (1, 4896), (300, 3000), (2600, 2600)])
def test_a_calls_workspace_does_not_depend_on_earlier_ones(monkeypatch, q_rows, kv_rows):
    """Every two calls of one shape, one after the other: each gets the workspace that the library asks for it."""
    q = torch.empty(1, 16, q_rows, 64, dtype=F16)
    k = torch.empty(1, 16, kv_rows, 64, dtype=F16)
    one = torch.ones(1, dtype=I32)
    calls = [dict(), dict(causal=True), dict(q_lens=one), dict(kv_lens=one), dict(q_lens=one, kv_lens=one),
             dict(q_starts=one), dict(causal=True, prefix_lens=one), dict(slopes=torch.ones(16)), dict(softcap=3.0)]
    if q_rows == kv_rows:
        calls += [dict(doc_offsets=torch.zeros(2, dtype=I32)), dict(doc_offsets=torch.zeros(2, dtype=I32), causal=True)]
    passed = []
    monkeypatch.setattr(block, "_sizes", {})
    monkeypatch.setattr(block, "_call", lambda name, dev, packed, stream: passed.append(packed))
    monkeypatch.setattr(block, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    for first in calls:
        for second in calls:
            block._sizes.clear()
            for kw in (first, second):
                attention(q, k, k, **kw)
                packed = passed.pop()
                given = block._ATTN.unpack(packed)[28]
                assert given == block._fn("h3qk_attention_workspace_bytes")(packed), (list(first), list(second))


@pytest.mark.parametrize("masks,cut", [(dict(), True), (dict(causal=1), False), (dict(causal=1, prefix_lens=A), True),
                                       (dict(q_lens=A), False)])
def test_which_last_rounds_are_cut(masks, cut):
    """176 tiles: a round and a bit of them.  Causal tiles go longest first, and what is left at the end is short."""
    f = dict(dtype=h3qk.FP16, batch=1, heads=16, kv_heads=16, head_dim=64, causal=0, docs=0, reserved=0, scale=0.0,
             softcap=0.0, q_rows=2600, kv_rows=2600, q=A, k=A, v=A, out=A, lse=A, grad_out=0, grad_q=0, grad_k=0,
             grad_v=0, slopes=0, prefix_lens=0, doc_offsets=0, q_lens=0, kv_lens=0, q_starts=0, workspace=0,
             workspace_bytes=0)
    f.update(masks)
    size = block._fn("h3qk_attention_workspace_bytes")(block._ATTN.pack(*f.values(), *[0] * 24))
    assert (size > 0) == cut
