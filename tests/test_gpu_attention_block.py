"""The example block: its operators together, trained and serving, and its
gradient against binary64."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import attention_block as E  # noqa: E402
import block_util as B  # noqa: E402

pytestmark = pytest.mark.gpu


def test_it_learns_and_serves():
    """The loss falls, and tokens taken one by one agree with the whole clip to the types' roundings: out is rounded
    twice to bf16 (2^-8 each) on either way."""
    losses, off = E.main(["--steps", "20", "--lengths", "130", "48", "200"])
    assert losses[-1] < 0.8 * losses[0]
    assert off < 4 * 2.0 ** -8


def test_its_gradient_against_binary64():
    """A whole block in fp16 against autograd on its definition in binary64.  Each of about ten stages rounds to 11
    bits; errors of independent roundings add as their squares, and 16 x 2^-11 leaves room for the correlated ones."""
    torch.manual_seed(1)
    block = E.Block(heads=3, dim=64, rotary=48, dtype=torch.float16)
    lengths = [70, 1, 150]
    n, c = sum(lengths), 192
    x = torch.randn(n, c, device="cuda").half().requires_grad_()
    pos = E.clip_positions(lengths)
    offsets = [0, 70, 71, 221]
    dout = torch.randn(n, c, device="cuda").half()
    masks = dict(causal=True, softcap=20.0, doc_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    out = block(x, pos, **masks)
    out.backward(dout)
    got = {"x": x.grad, **{k: p.grad for k, p in block.named_parameters()}}

    par = {k: (p.detach().half() if k in ("qkv", "out") else p.detach()).double().requires_grad_()
           for k, p in block.named_parameters()}
    xd = x.detach().double().requires_grad_()
    mean, var = xd.mean(1, keepdim=True), xd.var(1, unbiased=False, keepdim=True)
    y = (xd - mean) / (var + 1e-6).sqrt() * par["gain"] + par["shift"]
    rows = (y @ par["qkv"]).reshape(n, 3, 3, 64)
    ang = B.angles(pos, 48, (16, 16, 16))
    q, k = (B.norm_rope(rows[:, t], par[w], ang, 1e-6, 48).transpose(0, 1) for t, w in ((0, "wq"), (1, "wk")))
    v = rows[:, 2].transpose(0, 1)
    vis, _ = B.visible(n, n, 1, causal=True, doc_offsets=offsets)
    s = 20.0 * torch.tanh((q @ k.transpose(1, 2)) / 8.0 / 20.0)
    o = torch.softmax(s.masked_fill(~vis, -float("inf")), 2) @ v
    want = xd + o.transpose(0, 1).reshape(n, c) @ par["out"]
    want.backward(dout.double())
    B.assert_rel(out, want.detach(), 16 * 2.0 ** -11, "out")
    for name, g in got.items():
        B.assert_rel(g, (xd if name == "x" else par[name]).grad, 16 * 2.0 ** -11, name)


@pytest.mark.parametrize("raw", [False, True])
def test_workspaces_belong_to_the_stream_of_the_call(raw):
    """Calls on a side stream without workspaces of their own, while the current stream takes and fills memory."""
    from video_vae_decoder_qkv_gb300 import attention, attention_backward, layer_norm, layer_norm_backward

    q, k, v = (torch.randn(1, 8, 1500, 64, device="cuda").half() for _ in range(3))
    token, dout = q[:, :, :1].contiguous(), torch.randn_like(q)
    x, w = torch.randn(4000, 640, device="cuda").half(), torch.ones(640, device="cuda")

    def all_of(**kw):
        out, lse = attention(q, k, v, **kw)
        one = attention(token, k, v, **kw)
        _, stats = layer_norm(x, w, w, **kw)
        return [out, lse, *one, *attention_backward(dout, q, k, v, out, lse, **kw), *layer_norm_backward(x, x, w, stats, **kw)]

    want = all_of()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append(all_of(stream=side.cuda_stream if raw else side))
        for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22):
            torch.empty(n, device="cuda").fill_(float("nan"))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
