"""A pre-norm attention block on this package's operators: trained for a few
steps on packed clips, then asked for tokens one by one.

    python examples/attention_block.py [--steps N] [--width heads*dim] ...

The block is  x + W_out attention(prepare(W_qkv layer_norm(x))).  The two
projections are torch matrix products; every other step, forward and
backward, is one of the package's CUDA operators:

    layer_norm -> (W_qkv) -> prepare -> attention -> (W_out)
    layer_norm_backward <- ... <- prepare_backward <- attention_backward

Training packs clips of different lengths along the rows: each attends within
itself, causally after a prefix that all of its tokens see.  Serving fills a
cache with a clip's keys and values and appends one token at a time.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from video_vae_decoder_qkv_gb300 import (attention, attention_backward, layer_norm, layer_norm_backward,  # noqa: E402
                                         prepare, prepare_backward)


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, stats = layer_norm(x, weight, bias)
        ctx.save_for_backward(x, weight, stats)
        return y

    @staticmethod
    def backward(ctx, dy):
        return layer_norm_backward(dy.contiguous(), *ctx.saved_tensors)


class Prepare(torch.autograd.Function):
    """Per-head norm and rotary positions of the packed projection."""

    @staticmethod
    def forward(ctx, qkv, wq, wk, positions, sizes):
        q, k, v, _ = prepare(qkv, wq, wk, positions, **sizes)
        ctx.save_for_backward(qkv, wq, wk, positions)
        ctx.sizes = sizes
        return q, k, v

    @staticmethod
    def backward(ctx, dq, dk, dv):
        dqkv, dwq, dwk = prepare_backward(dq.contiguous(), dk.contiguous(), dv.contiguous(), *ctx.saved_tensors,
                                          **ctx.sizes)
        return dqkv, dwq, dwk, None, None


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, masks):
        # rows leave token-major, as the output projection reads them
        rows = torch.empty((q.shape[0], q.shape[2], q.shape[1], q.shape[3]), dtype=q.dtype, device=q.device)
        out, lse = attention(q, k, v, out=rows.transpose(1, 2), **masks)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.masks = masks
        return out

    @staticmethod
    def backward(ctx, dout):
        return *attention_backward(dout, *ctx.saved_tensors, **ctx.masks), None


class Block(torch.nn.Module):
    def __init__(self, heads=4, dim=64, rotary=48, dtype=torch.bfloat16):
        super().__init__()
        c = heads * dim
        par = lambda *s, scale=1.0: torch.nn.Parameter(scale * torch.randn(*s, device="cuda"))  # noqa: E731
        self.heads, self.dim, self.rotary, self.dtype = heads, dim, rotary, dtype
        self.gain, self.shift = torch.nn.Parameter(torch.ones(c, device="cuda")), par(c, scale=0.0)
        self.qkv, self.out = par(c, 3 * c, scale=c ** -0.5), par(c, c, scale=c ** -0.5)
        self.wq, self.wk = (torch.nn.Parameter(torch.ones(dim, device="cuda")) for _ in range(2))

    def heads_of(self, x, positions):
        y = Norm.apply(x, self.gain, self.shift)
        sizes = dict(heads=self.heads, head_dim=self.dim, rotary_dim=self.rotary)
        return Prepare.apply(y @ self.qkv.to(self.dtype), self.wq, self.wk, positions, sizes)

    def finish(self, x, rows):
        rows = rows.transpose(1, 2).reshape(x.shape[0], -1)
        return x + rows @ self.out.to(self.dtype)

    def forward(self, x, positions, **masks):
        return self.finish(x, Attention.apply(*self.heads_of(x, positions), masks))


class Cache:
    """Keys and values of one clip, filled from the front."""

    def __init__(self, block, room):
        shape = (1, block.heads, room, block.dim)
        self.k = torch.empty(shape, dtype=block.dtype, device="cuda")
        self.v = torch.empty(shape, dtype=block.dtype, device="cuda")
        self.length = 0

    def append(self, k, v):
        n = k.shape[2]
        self.k[:, :, self.length:self.length + n] = k
        self.v[:, :, self.length:self.length + n] = v
        self.length += n


@torch.no_grad()
def step(block, cache, x, positions, softcap=0.0):
    """The block on the next rows of a clip whose earlier ones are in the cache."""
    q, k, v = block.heads_of(x, positions)
    cache.append(k, v)
    lens = torch.tensor([cache.length], dtype=torch.int32, device="cuda")
    start = torch.tensor([cache.length - x.shape[0]], dtype=torch.int32, device="cuda")
    out, _ = attention(q, cache.k, cache.v, causal=True, kv_lens=lens, q_starts=start, softcap=softcap)
    return block.finish(x, out)


def clip_positions(lengths, wide=6):
    """(t, h, w) of each token on its clip's own grid, rows of `wide` tokens."""
    p = []
    for n in lengths:
        i = torch.arange(n)
        p.append(torch.stack([i // (4 * wide), i // wide % 4, i % wide], 1))
    return torch.cat(p).to(torch.int32).cuda()


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--dim", type=int, default=64)
    ap.add_argument("--lengths", type=int, nargs="+", default=[130, 48, 333])
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    block = Block(a.heads, a.dim, a.dim * 3 // 4 // 6 * 6)
    total, c = sum(a.lengths), a.heads * a.dim
    x = torch.randn(total, c, device="cuda").to(block.dtype)
    positions = clip_positions(a.lengths)
    offsets = torch.tensor([0, *torch.tensor(a.lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    prefixes = torch.tensor([n // 8 for n in a.lengths], dtype=torch.int32, device="cuda")
    masks = dict(causal=True, doc_offsets=offsets, prefix_lens=prefixes, softcap=30.0)
    # something to learn: each token's sum with the one before it, in its clip
    goal = x.float() + torch.roll(x.float(), 1, 0)
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    losses = []
    for i in range(a.steps):
        opt.zero_grad(set_to_none=True)
        loss = (block(x, positions, **masks).float() - goal).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps over clips of {a.lengths}")

    # one clip again, token by token after a first half in one call
    n, half = a.lengths[0], a.lengths[0] // 2
    clip, where = x[:n], positions[:n]
    with torch.no_grad():
        whole = block(clip, where, causal=True, softcap=30.0)
    cache = Cache(block, n + 7)
    parts = [step(block, cache, clip[:half], where[:half], 30.0)]
    parts += [step(block, cache, clip[i:i + 1], where[i:i + 1], 30.0) for i in range(half, n)]
    off = float((torch.cat(parts).float() - whole.float()).norm() / whole.float().norm())
    print(f"serving: {n - half} tokens one by one, {off:.2e} from the whole clip at once")
    return losses, off


if __name__ == "__main__":
    main()
