"""Attention forward against its definition in binary64 (block_util.attention
derives the bounds): sizes, types, shared heads, masks that leave rows empty,
layouts, and memory that nobody may read."""
import pytest

torch = pytest.importorskip("torch")

import block_util as B  # noqa: E402
from video_vae_decoder_qkv_gb300 import attention, block  # noqa: E402

pytestmark = pytest.mark.gpu


def _i32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def make(dtype, batch, heads, kv_heads, sq, sk, dim, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q = (gain * rnd(batch, heads, sq, dim)).to(dtype)
    k = (gain * rnd(batch, kv_heads, sk, dim)).to(dtype)
    v = rnd(batch, kv_heads, sk, dim)
    v[..., 0] *= 10
    return q, k, v.to(dtype)


def check(q, k, v, slopes=None, softcap=0.0, scale=None, **masks):
    lens = {n: _i32(x) if not isinstance(x, bool) else x for n, x in masks.items()}
    out, lse = attention(q, k, v, softcap=softcap, slopes=slopes, scale=scale, **lens)
    vis, dist = B.visible(q.shape[2], k.shape[2], q.shape[0], **masks)
    want = B.attention(q, k, v, vis, dist, softcap=softcap, slopes=slopes, scale=scale)
    empty = ~vis.any(2)[:, None].expand(lse.shape)
    assert (out[empty] == 0).all() and (lse[empty] == -float("inf")).all()
    B.assert_within(torch.where(empty, 0.0, lse), torch.where(empty, 0.0, want["lse"]), want["lse_bound"], "lse")
    B.assert_within(out, want["out"], want["out_bound"], "out")
    assert block._fn("h3qk_attention_stuck")() == 0
    return out, lse


TYPES = [torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("sq,sk", [(65, 65), (128, 128), (129, 257), (300, 100), (700, 701)])
def test_prompt_sizes(dtype, dim, sq, sk):
    check(*make(dtype, 1, 2, 2, sq, sk, dim))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("sq,sk", [(1, 1), (1, 2), (1, 127), (1, 4097), (3, 500), (16, 16), (64, 1000), (33, 64)])
def test_few_rows(dtype, dim, sq, sk):
    check(*make(dtype, 2, 2, 2, sq, sk, dim))
    check(*make(dtype, 1, 3, 3, sq, sk, dim, seed=1), causal=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (5, 1), (12, 12), (40, 8)])
@pytest.mark.parametrize("sq", [1, 4, 200])
def test_shared_heads(dtype, heads, kv_heads, sq):
    check(*make(dtype, 2, heads, kv_heads, sq, 300, 64), causal=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("s", [1, 90, 128, 300, 513])
def test_causal_and_prefix(dtype, dim, s):
    q, k, v = make(dtype, 2, 2, 1, s, s, dim)
    check(q, k, v, causal=True)
    check(q, k, v, causal=True, prefix_lens=[s // 3, s + 5])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sq,sk", [(1, 333), (7, 333), (150, 333), (333, 333)])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths_that_leave_rows_empty(dtype, sq, sk, causal):
    q, k, v = make(dtype, 4, 4, 2, sq, sk, 64, seed=2)
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


def test_many_documents():
    offsets = list(range(0, 1200, 13))
    check(*make(torch.bfloat16, 1, 2, 2, 1200, 1200, 64), doc_offsets=offsets)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sq,sk", [(1, 900), (2, 40), (400, 400)])
def test_capped_scores_and_distance(dtype, dim, sq, sk):
    q, k, v = make(dtype, 2, 4, 2, sq, sk, dim, gain=2.5)
    slopes = torch.tensor([0.5, 0.1, 0.01, -0.02], device="cuda")
    check(q, k, v, softcap=20.0)
    check(q, k, v, softcap=5.0, causal=True)
    check(q, k, v, slopes=slopes)
    check(q, k, v, slopes=slopes, softcap=30.0, causal=True, kv_lens=[sk, sk // 2 + 1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,sq,sk,dim,masks", [
    (2, 300, 3000, 64, {}),                                  # few tiles: all of them cut along the keys
    (3, 700, 2100, 128, dict(causal=True)),
    (16, 2600, 2600, 64, {}),                                # 176 tiles: a last round of 24
    (7, 1800, 1800, 72, dict(causal=True, prefix_lens=[700])),
    (2, 1700, 1700, 128, dict(q_lens=[1111], kv_lens=[1290])),
    (16, 2600, 2600, 64, dict(kv_lens=[2222])),
    (2, 300, 1500, 64, dict(kv_lens=[130])),                 # most parts without a key
    (2, 300, 1500, 64, dict(kv_lens=[0])),
    (4, 2000, 2000, 64, dict(doc_offsets=[0, 1100, 1101, 1500], causal=True)),
])
def test_tiles_cut_along_the_keys(dtype, heads, sq, sk, dim, masks):
    q, k, v = make(dtype, 1, heads, heads, sq, sk, dim, seed=8)
    offsets = masks.get("doc_offsets")
    pointers = [0] * 11 + [q.data_ptr() if offsets else 0] + [0] * 4  # doc_offsets alone is looked at
    call = block._ATTN.pack(block._DTYPES[dtype], 1, heads, heads, dim, 0, len(offsets) - 1 if offsets else 0, 0, 0.0, 0.0,
                            sq, sk, *pointers, 0, *[0] * 24)
    assert block._fn("h3qk_attention_workspace_bytes")(call) > 0
    check(q, k, v, **masks)
    check(q, k, v, softcap=15.0, slopes=torch.linspace(0.01, 0.3, heads, device="cuda"), **masks)


@pytest.mark.parametrize("sq", [1, 300])
def test_scores_far_apart(sq):
    """Rows whose weights sit on one key, or are all alike, or rise along the keys (the maximum keeps moving)."""
    q, k, v = make(torch.float16, 1, 2, 2, sq, 1500, 64)
    check(q * 8, k, v)
    check(q * 0, k, v)
    ramp = torch.linspace(-8, 8, 1500, device="cuda").to(k.dtype).view(1, 1, -1, 1)
    check(q.abs(), (k.abs() * ramp / 4).to(k.dtype), v)
    check(q, k, v, scale=0.7)


@pytest.mark.parametrize("sq", [2, 200])
def test_layouts(sq):
    b, h, hk, s, d = 2, 4, 2, 260, 64
    # token-major tensors, and heads inside a packed projection
    packed = torch.randn(b, s, (h + 2 * hk) * d + 8, device="cuda").to(torch.bfloat16)
    q = packed[..., :h * d].unflatten(2, (h, d)).transpose(1, 2)[:, :, :sq]
    k = packed[..., h * d:(h + hk) * d].unflatten(2, (hk, d)).transpose(1, 2)
    v = packed[..., (h + hk) * d:(h + 2 * hk) * d].unflatten(2, (hk, d)).transpose(1, 2)
    out, lse = check(q, k, v)
    plain = attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    # into the caller's own token-major rows
    mine = torch.full((b, sq, h, d + 8), 3.0, device="cuda", dtype=torch.bfloat16)
    got, _ = attention(q, k, v, out=mine[..., :d].transpose(1, 2))
    assert torch.equal(got, out) and (mine[..., d:] == 3).all()


@pytest.mark.parametrize("sq", [1, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 65504.0])
def test_unwritten_cache_rows_leave_no_mark(sq, bad):
    q, k, v = make(torch.float16, 3, 2, 2, sq, 1024, 64)
    lens = _i32([1000, 129, 640])
    want = attention(q, k, v, kv_lens=lens)
    for b, n in enumerate((1000, 129, 640)):
        k[b, :, n:] = bad
        v[b, :, n:] = bad
    got = attention(q, k, v, kv_lens=lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_documents_do_not_leak():
    q, k, v = make(torch.bfloat16, 1, 2, 2, 600, 600, 128)
    offsets = _i32([0, 130, 200, 470])
    want = attention(q, k, v, doc_offsets=offsets)
    for t in (q, k, v):
        t[:, :, 130:200] = float("nan")
        t[:, :, 470:] = float("inf")
    got = attention(q, k, v, doc_offsets=offsets)
    keep = [*range(130), *range(200, 600)]
    assert torch.equal(got[0][:, :, keep], want[0][:, :, keep]) and torch.equal(got[1][:, :, keep], want[1][:, :, keep])
    assert got[0][:, :, 130:200].isnan().all()


@pytest.mark.parametrize("sq", [1, 200])
def test_later_tokens_of_a_tile_do_not_leak_backwards_past_the_block(sq):
    q, k, v = make(torch.float16, 1, 1, 1, sq, 512, 64)
    want = attention(q, k, v, causal=True, q_starts=_i32([0]))
    k[:, :, sq:], v[:, :, sq:] = float("nan"), float("nan")
    got = attention(q, k, v, causal=True, q_starts=_i32([0]))
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("sq", [1, 130])
def test_a_visible_nan_is_passed_on(sq):
    q, k, v = make(torch.float16, 1, 2, 2, sq, 300, 64)
    k[0, 1, 77, 5] = float("nan")
    out, lse = attention(q, k, v)
    assert out[0, 1].isnan().all() and lse[0, 1].isnan().all()
    assert out[0, 0].isfinite().all() and lse[0, 0].isfinite().all()


@pytest.mark.parametrize("sq", [1, 200])
def test_a_cache_beyond_32_bit_offsets(sq):
    b, h, n, d = 2, 1, 300, 64
    stride = (1 << 32) + 64  # elements from item to item
    free = torch.cuda.mem_get_info()[0]
    if free < 24 << 30:
        pytest.skip("needs 24 GiB")
    q, k, v = make(torch.float16, b, h, h, sq, n, d)
    big = torch.empty(stride + 4 * n * d, dtype=torch.float16, device="cuda")
    kb = torch.as_strided(big, (b, h, n, d), (stride, n * d, d, 1), 0)
    vb = torch.as_strided(big, (b, h, n, d), (stride, n * d, d, 1), 2 * n * d)
    kb.copy_(k)
    vb.copy_(v)
    got, want = attention(q, kb, vb), attention(q, k, v)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("sq", [1, 300])
def test_stream_graph_and_caller_buffers(sq):
    q, k, v = make(torch.bfloat16, 2, 4, 2, sq, 2000, 128)
    lens = _i32([2000, 1100])
    want = attention(q, k, v, causal=True, kv_lens=lens)
    again = attention(q, k, v, causal=True, kv_lens=lens)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        attention(q, k, v, causal=True, kv_lens=lens, out=out, lse=lse, workspace=ws, stream=side)
    for _ in range(2):
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_no_rows_or_no_keys():
    q, k, v = make(torch.float16, 2, 2, 2, 0, 40, 64)
    out, lse = attention(q, k, v)
    assert out.shape == (2, 2, 0, 64) and lse.shape == (2, 2, 0)
    for sq in (1, 300):
        q, k, v = make(torch.float16, 2, 2, 2, sq, 0, 64)
        out, lse = attention(q, k, v)
        assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("ragged_first", [True, False])
def test_ragged_and_full_calls_of_one_shape(ragged_first):
    """More tiles than SMs, where lengths on the device decide about the workspace."""
    q, k, v = make(torch.float16, 1, 16, 16, 2600, 2600, 64, seed=4)
    block._sizes.clear()
    for ragged in (ragged_first, not ragged_first):
        check(q, k, v, **(dict(q_lens=[2311], kv_lens=[2400]) if ragged else {}))


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("sq,dim", [(1, 64), (300, 64), (300, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unwritten_cache_rows_leave_no_mark_on_capped_scores(sq, dim, bad, slopes):
    """Lengths that end 1, 2 and 3 past a multiple of 4."""
    q, k, v = make(torch.float16, 3, 2, 2, sq, 1024, dim)
    ends = (1001, 130, 643)
    kw = dict(kv_lens=_i32(ends), softcap=20.0, slopes=torch.tensor([0.1, 0.01], device="cuda") if slopes else None)
    want = attention(q, k, v, **kw)
    assert want[0].isfinite().all()
    for b, n in enumerate(ends):
        k[b, :, n:] = bad
        v[b, :, n:] = bad
    got = attention(q, k, v, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("causal", [False, True])
def test_documents_do_not_leak_into_capped_scores(causal):
    q, k, v = make(torch.bfloat16, 1, 2, 2, 600, 600, 128)
    kw = dict(doc_offsets=_i32([0, 130, 201, 472]), softcap=20.0, causal=causal)
    want = attention(q, k, v, **kw)
    for t in (q, k, v):
        t[:, :, 130:201] = float("nan")
        t[:, :, 472:] = float("inf")
    got = attention(q, k, v, **kw)
    keep = [*range(130), *range(201, 600)]
    assert torch.equal(got[0][:, :, keep], want[0][:, :, keep]) and torch.equal(got[1][:, :, keep], want[1][:, :, keep])
    assert got[0][:, :, 130:201].isnan().all()


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_a_key_concerns_only_the_rows_that_see_it(softcap):
    """A NaN in a key: its own and later rows, none before."""
    q, k, v = make(torch.float16, 1, 2, 2, 300, 300, 64)
    want = attention(q, k, v, causal=True, softcap=softcap)
    k[:, :, 77] = float("nan")
    got = attention(q, k, v, causal=True, softcap=softcap)
    assert torch.equal(got[0][:, :, :77], want[0][:, :, :77]) and torch.equal(got[1][:, :, :77], want[1][:, :, :77])
    assert got[0][:, :, 77:].isnan().all()


@pytest.mark.parametrize("sq", [1, 300])
def test_distances_past_24_bits(sq):
    """Positions that binary32 cannot hold, whose distances it can."""
    n, near = (1 << 24) + 40, 2000
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(1, 1, n, 8, generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    q = torch.randn(1, 2, sq, 8, generator=g, device="cuda", dtype=torch.float16)
    slopes = torch.tensor([0.5, 1.0], device="cuda")
    got = attention(q, k, v, slopes=slopes, causal=True)
    # what is further away than `near` weighs less than e^-800
    vis, dist = B.visible(sq, near, 1, causal=True)
    want = B.attention(q, k[:, :, n - near:], v[:, :, n - near:], vis, dist, slopes=slopes)
    B.assert_within(got[1], want["lse"], want["lse_bound"], "lse")
    B.assert_within(got[0], want["out"], want["out_bound"], "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sq,dim", [(1, 64), (300, 64), (300, 128)])
@pytest.mark.parametrize("softcap,gain", [(1025.0, 1.0), (1025.0, 8.0), (3e4, 1.0), (1e6, 1.0), (1e6, 4.0), (1e30, 1.0)])
def test_large_caps(dtype, sq, dim, softcap, gain):
    """A cap far above the scores leaves them their digits: the scores' bounds without the cap's share."""
    q, k, v = make(dtype, 1, 2, 2, sq, 700, dim, seed=15, gain=gain)
    slopes = torch.tensor([0.02, 0.0], device="cuda")
    vis, dist = B.visible(sq, 700, 1)
    for s in (None, slopes):
        out, lse = attention(q, k, v, softcap=softcap, slopes=s)
        want = B.attention(q, k, v, vis, dist, softcap=softcap, slopes=s)
        bound = B.attention(q, k, v, vis, dist, slopes=s)
        B.assert_within(lse, want["lse"], bound["lse_bound"], "lse")
        B.assert_within(out, want["out"], bound["out_bound"], "out")


@pytest.mark.parametrize("sq", [1, 300])
@pytest.mark.parametrize("softcap", [1e-3, 1e-30, 1e-38, 1e-40])
def test_small_caps(sq, softcap):
    """A cap far below the scores makes all weights alike, those of scores of 0 too."""
    q, k, v = make(torch.float16, 1, 2, 2, sq, 300, 64, seed=16)
    k[:, :, ::5] = 0
    check(q, k, v, softcap=softcap)
