"""Attention over a paged cache against binary64: formats, lengths, masks,
layouts of pools and rows, and how it is called."""
import math

import block_util as bu
import cache_util as cu
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from video_vae_decoder_qkv_gb300 import Cache, cache_attention  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16
SEQS = {
    "one": [(1, 1)], "page": [(1, 64)], "page+1": [(1, 65)], "tile": [(1, 1000)],
    "tokens": [(1, 130), (1, 1), (0, 77), (1, 0), (1, 700), (1, 16)],
    "drafts": [(4, 300), (3, 3), (0, 0), (5, 2000), (2, 17)],
    "rows16": [(3, 64), (8, 1111)], "rows40": [(7, 200), (40, 40), (13, 515)],
    "long": [(1, 40000)], "mixed": [(1, 3000), (300, 300), (1, 5), (129, 1000), (2, 4000), (0, 9), (64, 64)],
    "chunk": [(600, 1500)], "few of many": [(1, 40 * (i % 7)) for i in range(70)],
}


def run(seqs, dtype, fmt, heads, kv, dim, page, *, seed=1, causal=True, prefix=False, softcap=0.0, slopes=False, scale=None,
        k_scale=1.0, v_scale=1.0, layout="head", strided=False, tail=0, hint=True, mutate=None, q_times=1.0):
    rows, lens = [s[0] for s in seqs], [s[1] for s in seqs]
    cache, table, kv_lens = cu.build(lens, kv, dim, page, fmt, seed=seed, k_scale=k_scale, v_scale=v_scale, layout=layout)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    offsets = [0]
    for n in rows:
        offsets.append(offsets[-1] + n)
    tokens = offsets[-1] + tail
    q = (torch.randn(tokens, heads, dim, generator=g, device="cuda") * q_times / k_scale).to(dtype)
    if strided:
        wide = torch.full((tokens, heads + 3, dim + 8), math.nan, dtype=dtype, device="cuda")
        wide[:, 1:heads + 1, :dim] = q
        q = wide[:, 1:heads + 1, :dim]
    sl = torch.rand(heads, generator=g, device="cuda") * 0.2 if slopes else None
    pre = [n // 3 for n in lens] if prefix else None
    if mutate:
        mutate(cache, table, q)
    out = torch.full_like(q, 77.0)
    lse = torch.full((heads, tokens), 55.0, device="cuda")
    off_t = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    kw = dict(scale=scale, softcap=softcap, slopes=sl, causal=causal,
              prefix_lens=None if pre is None else torch.tensor(pre, dtype=torch.int32, device="cuda"))
    got = cache_attention(q, cache, table, kv_lens, q_offsets=off_t, max_rows=max(1, max(rows)) if hint else None, out=out,
                          lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    want, owned = cu.attention(q, cache, table, lens, offsets, causal=causal, prefix=pre, scale=scale, softcap=softcap,
                               slopes=sl)
    bu.assert_within(out[owned], want["out"][owned], want["out_bound"][owned], "out")
    mine, that = lse.t()[owned], want["lse"][owned]
    empty = torch.isneginf(that)
    assert torch.equal(torch.isneginf(mine), empty) and bool((out[owned][empty] == 0).all())
    bu.assert_within(mine[~empty], that[~empty], want["lse_bound"][owned][~empty], "lse")
    assert bool((out[~owned] == 77.0).all()) and bool((lse.t()[~owned] == 55.0).all())
    again = cache_attention(q, cache, table, kv_lens, q_offsets=off_t, max_rows=max(1, max(rows)) if hint else None,
                            out=torch.zeros_like(out), **kw)
    assert torch.equal(again[0][owned], out[owned]) and torch.equal(again[1].t()[owned], mine)
    return q, cache, table, kv_lens, off_t, out, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("seqs", list(SEQS))
def test_lengths(seqs, codes, dtype):
    run(SEQS[seqs], dtype, "e2m1" if codes else dtype, 10, 2, 64, 64)


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("seqs", ["tokens", "rows40", "chunk"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_dims_4bit(dim, seqs, dtype):
    run(SEQS[seqs], dtype, "e2m1", 4, 2, dim, 32)


@pytest.mark.parametrize("dim", [8, 40, 72, 128])
@pytest.mark.parametrize("seqs", ["tokens", "rows40", "chunk"])
def test_dims_16bit(dim, seqs):
    run(SEQS[seqs], BF16, BF16, 4, 2, dim, 32)


@pytest.mark.parametrize("page", [16, 32, 128, 512])
@pytest.mark.parametrize("fmt", ["e2m1", F16])
@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
def test_pages(page, fmt, seqs):
    run(SEQS[seqs], F16, fmt, 8, 2, 128, page)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (16, 1), (40, 8), (7, 1), (34, 2)])
@pytest.mark.parametrize("fmt", ["e2m1", BF16])
@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
def test_heads(heads, kv, fmt, seqs):
    run(SEQS[seqs], BF16, fmt, heads, kv, 64, 64)


@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(prefix=True), dict(softcap=5.0), dict(softcap=3000.0), dict(slopes=True),
    dict(softcap=30.0, slopes=True, prefix=True), dict(scale=0.5), dict(causal=False, softcap=20.0, slopes=True),
], ids=lambda k: "-".join(k))
@pytest.mark.parametrize("fmt", ["e2m1", BF16])
@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
def test_masks_and_bends(kw, fmt, seqs):
    run(SEQS[seqs], BF16, fmt, 10, 2, 128, 64, **kw)


@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
@pytest.mark.parametrize("k_scale,v_scale", [(0.37, 11.0), (2.0 ** -12, 300.0)])
def test_tensor_scales(seqs, k_scale, v_scale):
    run(SEQS[seqs], F16 if k_scale > 0.1 else BF16, "e2m1", 10, 2, 64, 64, k_scale=k_scale, v_scale=v_scale)


@pytest.mark.parametrize("times", [1e-25, 1e-3, 1e15])
def test_rows_of_any_size_keep_their_digits(times):
    """bfloat16 rows far from 1, with the scale that makes their scores ordinary."""
    run(SEQS["drafts"], BF16, "e2m1", 10, 2, 64, 64, q_times=times, scale=0.1 / times)


@pytest.mark.parametrize("fmt", ["e2m1", F16])
@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
def test_strided_rows_and_rows_of_no_sequence(fmt, seqs):
    run(SEQS[seqs], F16, fmt, 10, 2, 64, 64, strided=True, tail=9, hint=False)


@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
def test_pool_of_rows_with_heads_beside_each_other(seqs):
    run(SEQS[seqs], BF16, BF16, 10, 2, 72, 64, layout="row")


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
@pytest.mark.parametrize("seqs", ["drafts", "mixed"])
def test_pages_outside_the_pool_read_as_zeros(fmt, seqs):
    def mutate(cache, table, q):
        table[0, 0] = -1
        table[-1, 0] = cache.pages
        table[3, -1] = 2 ** 31 - 1

    run(SEQS[seqs], BF16, fmt, 10, 2, 64, 16, mutate=mutate)


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
@pytest.mark.parametrize("rows", [1, 60])
def test_rows_without_offsets(fmt, rows):
    cache, table, lens = cu.build([100, 61, 400], 2, 64, 32, fmt)
    q = torch.randn(3 * rows, 4, 64, device="cuda").to(BF16)
    off = torch.arange(0, 3 * rows + 1, rows, dtype=torch.int32, device="cuda")
    a, b = cache_attention(q, cache, table, lens), cache_attention(q, cache, table, lens, q_offsets=off, max_rows=rows)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # without max_rows the host does not know the sequences' rows, and may cut the call otherwise
    c = cache_attention(q, cache, table, lens, q_offsets=off)
    want, _ = cu.attention(q, cache, table, lens.tolist(), off.tolist())
    for got in (a, c):
        bu.assert_within(got[0], want["out"], want["out_bound"], "out")


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
@pytest.mark.parametrize("rows,most", [(5, 2), (90, 60)])
def test_rows_past_max_rows_are_left(fmt, rows, most):
    """A sequence's first rows keep their places; the later ones are not touched."""
    cache, table, lens = cu.build([rows, 300], 2, 64, 32, fmt)
    q = torch.randn(2 * rows, 4, 64, device="cuda").to(BF16)
    out = torch.full_like(q, 9.0)
    cache_attention(q, cache, table, lens, max_rows=most, out=out)
    want, _ = cu.attention(q, cache, table, lens.tolist(), [0, rows, 2 * rows])
    kept = (torch.arange(2 * rows) % rows) < most
    bu.assert_within(out[kept], want["out"][kept], want["out_bound"][kept], "out")
    assert bool((out[~kept] == 9.0).all())


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_call_on_a_device_that_is_not_current(fmt):
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    cache, table, lens = cu.build([200], 2, 64, 32, fmt)
    q = torch.randn(1, 4, 64, device="cuda:0").to(BF16)
    want = cache_attention(q, cache, table, lens)
    with torch.cuda.device(1):
        got = cache_attention(q, cache, table, lens)
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_empty_pool_and_empty_table(fmt, rows):
    """No pages at all: every row sees zeros where it has keys, and nothing where the table has no room."""
    cache = Cache.empty(0, 2, 64, dtype=fmt)
    q = torch.randn(2 * rows, 4, 64, device="cuda").to(BF16)
    lens = torch.tensor([rows, 0], dtype=torch.int32, device="cuda")
    out, lse = cache_attention(q, cache, torch.zeros(2, 8, dtype=torch.int32, device="cuda"), lens)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse[:, rows:]).all())
    n = torch.arange(1, rows + 1, device="cuda").clamp(max=512)
    assert torch.allclose(lse[0, :rows], n.float().log(), atol=1e-5)
    out, lse = cache_attention(q, cache, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), lens)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_nan_reaches_only_the_rows_that_see_it(fmt):
    for rows in (3, 70):
        cache, table, lens = cu.build([500, 500], 1, 64, 64, fmt)
        at = (int(table[0, 490 // 64]), 0, 490 % 64)
        if fmt == "e2m1":
            cache.k_scales.view(torch.uint8)[at] = 0x7F
        else:
            cache.k[at] = math.nan
        q = torch.randn(2 * rows, 2, 64, device="cuda").to(BF16)
        out, lse = cache_attention(q, cache, table, lens, causal=True)
        sees = torch.arange(500 - rows, 500, device="cuda") >= 490
        assert torch.equal(torch.isnan(out[:rows]).any(2).any(1), sees)
        assert torch.equal(torch.isnan(lse[:, :rows]).any(0), sees)
        assert not torch.isnan(out[rows:]).any()


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_lengths_beyond_the_table_are_cut(fmt):
    cache, table, lens = cu.build([128, 128], 2, 64, 64, fmt)
    q = torch.randn(2, 4, 64, device="cuda").to(BF16)
    want = cache_attention(q, cache, table, lens)
    lens[0] = 2 ** 31 - 1
    got = cache_attention(q, cache, table, lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    lens[1] = -5
    got = cache_attention(q, cache, table, lens)
    assert bool((got[0][1] == 0).all()) and bool(torch.isneginf(got[1][:, 1]).all())


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_captured_calls_follow_their_lists(fmt):
    """One captured call serves a cache that grows: lengths and pages are read on the device."""
    cache, table, lens = cu.build([900, 700, 64, 1], 2, 64, 64, fmt)
    q = torch.randn(4, 10, 64, device="cuda").to(BF16)
    full, lens_now, out = lens.clone(), lens.clone(), torch.empty_like(q)
    lse = torch.empty(10, 4, device="cuda")
    cache_attention(q, cache, table, lens_now, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache_attention(q, cache, table, lens_now, out=out, lse=lse)
    for cut in (1, 2, 5):
        lens_now.copy_(full // cut)
        graph.replay()
        want = cache_attention(q, cache, table, lens_now)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_two_streams_at_once():
    sets = [cu.build([3000 + 500 * i, 800], 2, 128, 64, "e2m1", seed=i) for i in range(2)]
    qs = [torch.randn(2, 10, 128, device="cuda").to(BF16) for _ in range(2)]
    want = [cache_attention(q, *s)[0] for q, s in zip(qs, sets)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(cache_attention(qs[i], *sets[i], stream=streams[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            assert torch.equal(x, want[i])


def test_offsets_of_a_large_pool_pass_32_bits():
    """The last pages of a pool of more than 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough free memory")
    pages = 70000
    pool = torch.empty(2, pages, 4, 64, 128, dtype=BF16, device="cuda")
    small, table, lens = cu.build([200, 300], 4, 128, 64, BF16)
    far = (pages - 1 - torch.arange(small.pages, device="cuda"))
    pool[0, far], pool[1, far] = small.k, small.v
    q = torch.randn(2, 8, 128, device="cuda").to(BF16)
    want = cache_attention(q, small, table, lens)
    got = cache_attention(q, Cache(pool[0], pool[1]), far[table.long()].int(), lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_block_gave_up():
    """After everything above: the kernels' bounded waits never ran out."""
    from video_vae_decoder_qkv_gb300 import block

    assert block._fn("h3qk_attention_stuck")() == 0
