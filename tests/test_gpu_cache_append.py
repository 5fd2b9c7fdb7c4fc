"""Appending to a paged cache and reading it back: bit for bit what `prepare`
writes, and its 4-bit codes; and a run of the cache's operators together."""
import math

import block_util as bu
import cache_util as cu
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from video_vae_decoder_qkv_gb300 import (Cache, attention, cache_append, cache_attention, cache_read,  # noqa: E402
                                         prepare)

F16, BF16 = torch.float16, torch.bfloat16


def prepared(qkv, wq, wk, pos, heads, kv, dim, rotary, axes):
    """Q, K, V [tokens, heads, dim] by `prepare`, which has as many K/V heads as heads."""
    tokens = qkv.shape[0]
    n = max(heads, kv)
    x = qkv[:, :(heads + 2 * kv) * dim].reshape(tokens, heads + 2 * kv, dim)
    wide = torch.zeros(tokens, 3, n, dim, dtype=qkv.dtype, device="cuda")
    wide[:, 0, :heads], wide[:, 1, :kv], wide[:, 2, :kv] = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    q, k, v, _ = prepare(wide.view(tokens, -1), wq, wk, pos, heads=n, head_dim=dim, rotary_dim=rotary, n_axes=axes,
                         out_layout="token_major")
    q, k, v = (t.view(tokens, n, dim) for t in (q, k, v))
    return q[:, :heads], k[:, :kv], v[:, :kv]


def expected(cache, table, lens, offsets, k, v):
    """The pool after the append: bytes of k, v (and scales)."""
    parts = [t.clone() for t in (cache.k, cache.v)]
    scales = [None if t is None else t.view(torch.uint8).clone() for t in (cache.k_scales, cache.v_scales)]
    page = cache.page_size
    for b, keys in enumerate(lens):
        n = offsets[b + 1] - offsets[b]
        for i in range(n):
            at = keys - n + i
            if at < 0 or at // page >= table.shape[1]:
                continue
            pg = int(table[b, at // page])
            if not 0 <= pg < cache.pages:
                continue
            for t, (x, ts) in enumerate(((k, cache.k_scale), (v, cache.v_scale))):
                row = x[offsets[b] + i]
                if scales[t] is None:
                    parts[t][pg, :, at % page] = row
                else:
                    codes, by = cu.encode(row, ts)
                    parts[t][pg, :, at % page] = cu.pack(codes)
                    scales[t][pg, :, at % page] = by
    return parts, scales


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check(seqs, dtype, fmt, heads, kv, dim, page, *, rotary=None, axes=1, give=False, layout="head", k_scale=1.0, v_scale=1.0,
          pad=0, tail=0, mutate=None, edit=None, offsets=None):
    rows, lens = [s[0] for s in seqs], [s[1] for s in seqs]
    cache, table, kv_lens = cu.build([max(0, n) for n in lens], kv, dim, page, fmt, layout=layout, k_scale=k_scale,
                                     v_scale=v_scale)
    g = torch.Generator(device="cuda").manual_seed(5)
    if offsets is None:
        offsets = [0]
        for n in rows:
            offsets.append(offsets[-1] + n)
    tokens = offsets[-1] + tail
    rotary = dim if rotary is None else rotary
    qkv = torch.randn(tokens, (heads + 2 * kv) * dim + pad, generator=g, device="cuda").to(dtype)
    qkv[:, :(heads + 2 * kv) * dim] *= torch.exp2(torch.randint(-4, 4, (1, (heads + 2 * kv) * dim), generator=g,
                                                                device="cuda").float()).to(dtype)
    if edit:
        edit(qkv)
    wq, wk = (torch.rand(dim, generator=g, device="cuda") + 0.5 for _ in range(2))
    pos = torch.zeros(tokens, axes, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        m = offsets[b + 1] - offsets[b]
        pos[offsets[b]:offsets[b + 1], 0] = torch.arange(n - m, n, device="cuda", dtype=torch.int32)
    if give:
        pos += torch.randint(0, 60, pos.shape, generator=g, device="cuda", dtype=torch.int32)
    if mutate:
        mutate(cache, table)
    q, k, v = prepared(qkv, wq, wk, pos, heads, kv, dim, rotary, axes)
    parts, scales = expected(cache, table, lens, offsets, k, v)
    out = torch.full((tokens, heads, dim), 3.0, dtype=dtype, device="cuda")
    got = cache_append(qkv, wq, wk, cache, table, kv_lens if mutate is None else torch.tensor(lens, dtype=torch.int32).cuda(),
                       heads=heads, rotary_dim=rotary, positions=pos if give else None,
                       q_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    owned = torch.zeros(tokens, dtype=torch.bool)
    owned[offsets[0]:offsets[-1]] = True
    assert same_bytes(got[owned], q[owned]) and bool((got[~owned] == 3.0).all())
    for mine, want in ((cache.k, parts[0]), (cache.v, parts[1])):
        assert same_bytes(mine, want)
    for mine, want in ((cache.k_scales, scales[0]), (cache.v_scales, scales[1])):
        if mine is not None:
            assert torch.equal(mine.view(torch.uint8), want)
    return cache, table, kv_lens


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 65)], [(17, 40), (0, 9), (1, 70), (33, 33)], [(130, 500)]])
@pytest.mark.parametrize("dim", [32, 96, 128])
def test_append(seqs, codes, dtype, dim):
    check(seqs, dtype, "e2m1" if codes else dtype, 6, 2, dim, 32)


@pytest.mark.parametrize("dim,rotary,axes", [(8, 6, 3), (40, 24, 3), (72, 0, 1), (128, 96, 3), (64, 48, 3)])
def test_append_16bit_with_positions(dim, rotary, axes):
    check([(5, 20), (40, 41)], BF16, BF16, 4, 4, dim, 16, rotary=rotary, axes=axes, give=True, pad=16)


@pytest.mark.parametrize("dim,rotary,axes", [(32, 6, 3), (96, 0, 1), (128, 96, 3), (64, 48, 3)])
def test_append_4bit_with_positions(dim, rotary, axes):
    check([(5, 20), (40, 41)], F16, "e2m1", 3, 1, dim, 16, rotary=rotary, axes=axes, give=True, pad=16)


@pytest.mark.parametrize("k_scale,v_scale", [(0.37, 11.0), (2.0 ** -10, 100.0)])
def test_append_tensor_scales(k_scale, v_scale):
    check([(9, 20), (40, 41)], BF16, "e2m1", 4, 2, 64, 64, k_scale=k_scale, v_scale=v_scale)


def test_append_pool_of_rows_with_heads_beside_each_other():
    check([(9, 20), (40, 41)], F16, F16, 4, 2, 72, 32, layout="row")


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_rows_of_no_sequence_are_left(fmt):
    check([(9, 20), (40, 41)], BF16, fmt, 4, 2, 64, 32, tail=11)
    check([(9, 20), (40, 41)], BF16, fmt, 4, 2, 64, 32, tail=3, offsets=[4, 13, 53])


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_places_outside_the_table_or_the_pool_are_not_written(fmt):
    def mutate(cache, table):
        table[0, 0] = -1
        table[1, 0] = cache.pages
        table[1, 1] = 2 ** 31 - 1

    check([(9, 20), (60, 90), (5, 3), (40, 130)], BF16, fmt, 4, 2, 64, 32, mutate=mutate)


def test_values_that_are_not_finite_mark_their_group():
    def edit(qkv):
        at = 6 * 64  # V of two heads, after 4 + 2 of Q and K
        qkv[0, at + 3], qkv[1, at + 20], qkv[2, at + 70] = math.nan, math.inf, -math.inf
        qkv[3, at:] = 0
        qkv[4, at:] *= 1e-30
        qkv[5, at + 16:at + 32] = 3e38

    cache, table, lens = check([(8, 8)], BF16, "e2m1", 4, 2, 64, 32, edit=edit)
    _, v = cache_read(cache, table, lens, rows=8)
    assert torch.isnan(v[0, 0, 0, :16]).all() and not torch.isnan(v[0, 0, 0, 16:]).any()
    assert bool((v[0, :, 3] == 0).all()) and float(v[0, 0, 5, 16]) == 6 * 448


def test_rounding_of_4_bits_is_half_a_step():
    """|value - y| <= half the distance of neighbouring codes, times the group's scale (and a bound for its rounding)."""
    y = torch.randn(4096, 2, 128, device="cuda").to(BF16)
    w = torch.ones(128, device="cuda")
    cache = Cache.empty(64, 2, 128, dtype="e2m1")
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([4096], dtype=torch.int32, device="cuda")
    qkv = torch.cat([y[:, :1], y, y], 1).view(4096, -1)
    cache_append(qkv, w, w, cache, table, lens, heads=1, rotary_dim=0)
    _, v = cache_read(cache, table, lens, dtype=BF16)
    v, y = v[0].transpose(0, 1).double().unflatten(-1, (-1, 16)), y.double().unflatten(-1, (-1, 16))
    top = y.abs().amax(-1, keepdim=True)
    # the scale is within 2^-4 of top / 6, so codes reach 6 / (1 - 2^-4); the widest gap between codes is 2
    assert bool(((v - y).abs() <= top / 6 * (1 + 2.0 ** -4) * torch.where(y.abs() * 6 > top * 4 * (1 - 2.0 ** -4), 1.0, 0.5)).all())


@pytest.mark.parametrize("fmt", ["e2m1", F16])
@pytest.mark.parametrize("dim", [32, 96, 128])
def test_read(fmt, dim):
    lens = [100, 0, 37, 64]
    cache, table, kv_lens = cu.build(lens, 3, dim, 32, fmt, k_scale=1.0 if fmt == F16 else 0.3,
                                     v_scale=1.0 if fmt == F16 else 7.0)
    table[2, 0] = -1
    k_all, v_all = cu.values(cache)
    starts = [0, 0, 30, 70]
    for s in (None, starts):
        for rows in (None, 1, 50, 300):
            st = None if s is None else torch.tensor(s, dtype=torch.int32, device="cuda")
            k, v = cache_read(cache, table, kv_lens, starts=st, rows=rows, dtype=F16)
            n = table.shape[1] * 32 if rows is None else rows
            for got, pool in ((k, k_all), (v, v_all)):
                want = torch.zeros(4, 3, n, dim, dtype=torch.float64, device="cuda")
                for b in range(4):
                    x = cu.rows_of(pool, table[b], lens[b])[:, 0 if s is None else s[b]:][:, :n]
                    want[b, :, :x.shape[1]] = x
                # rounded once to binary32, once to 16 bits
                bu.assert_within(got, want, want.abs() * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25, "read")


def test_read_of_codes_is_exact():
    cache, table, kv_lens = cu.build([200], 2, 64, 64, "e2m1")
    k_all, _ = cu.values(cache)
    for dtype in (F16, BF16):
        k, _ = cache_read(cache, table, kv_lens, rows=200, dtype=dtype)
        assert torch.equal(k[0].double(), cu.rows_of(k_all, table[0], 200))


@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_serving_run(fmt):
    """Prompts in chunks, then tokens one by one, for requests that come and go: the cache holds what `prepare` gives,
    and attention over it is attention over the whole sequences."""
    heads, kv, dim, page = 10, 2, 64, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = Cache.empty(40, kv, dim, page_size=page, dtype=fmt)
    free = list(range(40))
    table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    lens, seen = [0, 0, 0], [[], [], []]
    wq, wk = (torch.rand(dim, generator=g, device="cuda") + 0.5 for _ in range(2))
    steps = [[100, 0, 7], [64, 33, 1], [1, 1, 1], [1, 1, 1], [70, 1, 1], [1, 0, 1], [1, 130, 1]]
    for step, new in enumerate(steps):
        if step == 4:  # the first request ends; another takes its pages
            free += [int(x) for x in table[0] if int(x) >= 0]
            table[0] = -1
            lens[0], seen[0] = 0, []
        for b, n in enumerate(new):
            lens[b] += n
            for i in range(-(-lens[b] // page)):
                if int(table[b, i]) < 0:
                    table[b, i] = free.pop(0)
        tokens = sum(new)
        offsets = [0, new[0], new[0] + new[1], tokens]
        qkv = torch.randn(tokens, (heads + 2 * kv) * dim, generator=g, device="cuda").to(BF16)
        kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        q = cache_append(qkv, wq, wk, cache, table, kv_lens, heads=heads, rotary_dim=48, q_offsets=off)
        out, _ = cache_attention(q, cache, table, kv_lens, q_offsets=off)
        want, owned = cu.attention(q, cache, table, lens, offsets)
        bu.assert_within(out[owned], want["out"][owned], want["out_bound"][owned], f"step {step}")
        for b in range(3):
            seen[b].append(qkv[offsets[b]:offsets[b + 1]])
    k, v = cache_read(cache, table, kv_lens, rows=max(lens), dtype=BF16)
    for b in range(3):
        rows = torch.cat(seen[b])
        pos = torch.arange(lens[b], dtype=torch.int32, device="cuda")[:, None]
        _, kk, vv = prepared(rows, wq, wk, pos, heads, kv, dim, 48, 1)
        for got, x in ((k, kk), (v, vv)):
            if fmt == BF16:
                assert torch.equal(got[b, :, :lens[b]].transpose(0, 1), x)
            else:
                codes, by = cu.encode(x)
                want = cu.code_values(codes) * by.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
                assert torch.equal(got[b, :, :lens[b]].transpose(0, 1).double(), want)
    # the last tokens again, over the dense rows
    last = q[offsets[2]:offsets[3]]
    dense, _ = attention(last.transpose(0, 1)[None].contiguous(), k[2:, :, :lens[2]], v[2:, :, :lens[2]], causal=True)
    bound = want_bound(want=cu.attention(q, cache, table, lens, offsets)[0], rows=slice(offsets[2], offsets[3]))
    bu.assert_within(dense[0].transpose(0, 1), out[offsets[2]:offsets[3]].double(), 2 * bound, "dense")


def want_bound(want, rows):
    return want["out_bound"][rows]


def test_append_on_a_captured_stream():
    """A captured step follows the lengths and pages that are on the device when it is replayed."""
    cache, table, lens = cu.build([100, 60], 2, 64, 32, "e2m1", extra_pages=2)
    qkv = torch.randn(2, 8 * 64, device="cuda").to(BF16)
    w = torch.ones(64, device="cuda")
    out = torch.empty(2, 4, 64, dtype=BF16, device="cuda")
    att = torch.empty_like(out)
    lse = torch.empty(4, 2, device="cuda")

    def step():
        lens.add_(1)
        cache_append(qkv, w, w, cache, table, lens, heads=4, rotary_dim=64, out=out)
        cache_attention(out, cache, table, lens, out=att, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        qkv.copy_(torch.randn(2, 8 * 64, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        now = [101 + 1 + i, 61 + 1 + i]
        assert lens.tolist() == now
        want, _ = cu.attention(out, cache, table, now, [0, 1, 2])
        bu.assert_within(att, want["out"], want["out_bound"], "captured")
