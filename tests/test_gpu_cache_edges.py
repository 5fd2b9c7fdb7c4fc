"""The paged cache's operators where their documentation allows more than
ordinary calls make: rows that are not finite beside rows that are,
sequences that are longer than their table, the largest and smallest scales,
and what the 4-bit format's roundings are."""
import math

import block_util as bu
import cache_util as cu
import pytest
from test_gpu_cache_append import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from video_vae_decoder_qkv_gb300 import Cache, cache_append, cache_attention, cache_read, prepare  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16


def spoil(cache, table, item, key):
    """NaN in a sequence's key, of every K/V head."""
    page, at = int(table[item, key // cache.page_size]), key % cache.page_size
    if cache.dtype == "e2m1":
        cache.k_scales.view(torch.uint8)[page, :, at] = 0x7F
    else:
        cache.k[page, :, at] = math.nan


@pytest.mark.parametrize("softcap", [30.0, 2000.0])
@pytest.mark.parametrize("group", [1, 3, 5])
@pytest.mark.parametrize("rows", [2, 3, 4, 70])
@pytest.mark.parametrize("fmt,dtype", [("e2m1", BF16), (BF16, BF16), (F16, F16)])
def test_nan_key_under_a_cap_reaches_only_the_rows_that_see_it(fmt, dtype, rows, group, softcap):
    """The last key, which only the last row sees; the key 8 before it, with which it shares a lane, is seen by others."""
    kv, lens = 2, [510, 200]
    cache, table, kv_lens = cu.build(lens, kv, 64, 64, fmt)
    spoil(cache, table, 0, 509)
    q = torch.randn(2 * rows, kv * group, 64, device="cuda").to(dtype)
    out, lse = cache_attention(q, cache, table, kv_lens, softcap=softcap)
    want, _ = cu.attention(q, cache, table, lens, [0, rows, 2 * rows], softcap=softcap)
    sees = torch.zeros(2 * rows, dtype=torch.bool, device="cuda")
    sees[rows - 1] = True
    assert bool(torch.isnan(out[sees]).all()) and bool(torch.isnan(lse[:, sees]).all())
    bu.assert_within(out[~sees], want["out"][~sees], want["out_bound"][~sees], "out")
    bu.assert_within(lse.t()[~sees], want["lse"][~sees], want["lse_bound"][~sees], "lse")


@pytest.mark.parametrize("softcap", [0.0, 30.0, 2000.0])
@pytest.mark.parametrize("rows,group", [(1, 5), (1, 8), (3, 5), (70, 5)])
@pytest.mark.parametrize("fmt,dtype", [("e2m1", BF16), (BF16, BF16), (F16, F16)])
def test_nan_row_reaches_no_other(fmt, dtype, rows, group, softcap):
    kv, lens = 2, [300, 200]
    cache, table, kv_lens = cu.build(lens, kv, 64, 64, fmt)
    q = torch.randn(2 * rows, kv * group, 64, device="cuda").to(dtype)
    clean = q.clone()
    spoilt = torch.zeros(2 * rows, kv * group, dtype=torch.bool, device="cuda")
    spoilt[rows // 2, 1::3] = True
    q[spoilt] = math.nan
    out, lse = cache_attention(q, cache, table, kv_lens, softcap=softcap)
    want, _ = cu.attention(clean, cache, table, lens, [0, rows, 2 * rows], softcap=softcap)
    assert bool(torch.isnan(out[spoilt]).all()) and bool(torch.isnan(lse.t()[spoilt]).all())
    for got, name in ((out, "out"), (lse.t(), "lse")):
        bu.assert_within(got[~spoilt], want[name][~spoilt], want[name + "_bound"][~spoilt], name)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("rows,past", [(2, 1), (4, 2), (3, 900), (40, 2), (300, 37), (40, 2 ** 31 - 1 - 320)])
@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_rows_of_sequences_past_their_table_keep_their_positions(fmt, rows, past, slopes):
    """Row i stands at kv_lens - n + i, as the append places it, whatever the table has room for."""
    if slopes and past > 1000:
        pytest.skip("scores less a slope times 2^31 have no digits left")
    room, heads = 320, 4
    cache, table, kv_lens = cu.build([room, 100], 2, 64, 64, fmt)
    kv_lens[0] = room + past
    q = torch.randn(2 * rows, heads, 64, device="cuda").to(BF16)
    sl = torch.rand(heads, device="cuda") * 0.2 if slopes else None
    out, lse = cache_attention(q, cache, table, kv_lens, slopes=sl)
    k_all, v_all = cu.values(cache)
    for b, keys, start in ((0, room, room + past - rows), (1, 100, 100 - rows)):
        at = slice(b * rows, (b + 1) * rows)
        # (where a row stands past the keys, what it sees is all of them)
        vis, dist = bu.visible(rows, keys, 1, True, q_starts=[start])
        want = bu.attention(q[at].transpose(0, 1)[None], cu.rows_of(k_all, table[b], keys)[None],
                            cu.rows_of(v_all, table[b], keys)[None], vis, dist, slopes=sl)
        bu.assert_within(out[at].transpose(0, 1), want["out"][0], want["out_bound"][0], "out")
        seen = ~torch.isneginf(want["lse"][0])
        assert torch.equal(~torch.isneginf(lse[:, at]), seen)
        bu.assert_within(lse[:, at][seen], want["lse"][0][seen], want["lse_bound"][0][seen], "lse")


@pytest.mark.parametrize("length", [2 ** 30 + 5, 2 ** 31 - 1])
def test_places_past_2_30_turn_q_by_their_own_angle(length):
    cache, table, kv_lens = cu.build([64], 2, 64, 64, BF16)
    kv_lens[0] = length
    qkv = torch.randn(3, 6 * 64, device="cuda").to(BF16)
    w = torch.rand(64, device="cuda") + 0.5
    was = cache.k.clone(), cache.v.clone()
    got = cache_append(qkv, w, w, cache, table, kv_lens, heads=2, rotary_dim=64)
    pos = torch.arange(length - 3, length, device="cuda").int()[:, None]
    want = prepare(qkv, w, w, pos, heads=2, head_dim=64, rotary_dim=64, n_axes=1, out_layout="token_major")[0]
    assert torch.equal(got.flatten(), want.flatten())
    for now, then in zip((cache.k, cache.v), was):
        assert torch.equal(now.view(torch.int16), then.view(torch.int16))


@pytest.mark.parametrize("log2", [-117, 117])
def test_append_with_the_largest_and_smallest_tensor_scales(log2):
    """Values of the scale's size get their codes, and zeros stay zeros."""
    def edit(qkv):
        qkv[:, 6 * 64:] *= 2.0 ** log2  # V of two heads, after 4 + 2 of Q and K
        qkv[3, 6 * 64:] = 0

    cache, table, lens = check([(9, 20), (40, 41)], BF16, "e2m1", 4, 2, 64, 64, k_scale=1.0, v_scale=2.0 ** log2, edit=edit)
    _, v = cache_read(cache, table, lens, rows=20)
    assert bool((v[0, :, 14] == 0).all()) and bool(v[0, :, 15].any())


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("exponent,softcap", [(120, 1e-8), (100, 1e-20), (0, 1e-40)])
@pytest.mark.parametrize("fmt", ["e2m1", BF16])
def test_caps_far_below_the_scores(fmt, exponent, softcap, rows):
    """All that a row sees lies within +-softcap of 0, so that it weighs the same (to 2e-8, well below the bound's 2^-18)."""
    lens = [100, 70]
    cache, table, kv_lens = cu.build(lens, 1, 64, 64, fmt)
    q = (torch.randn(2 * rows, 2, 64, device="cuda") * 2.0 ** exponent).to(BF16)
    out, lse = cache_attention(q, cache, table, kv_lens, softcap=softcap)
    want, _ = cu.attention(torch.zeros_like(q), cache, table, lens, [0, rows, 2 * rows])
    bu.assert_within(out, want["out"], want["out_bound"], "out")
    bu.assert_within(lse.t(), want["lse"], want["lse_bound"], "lse")


@pytest.mark.parametrize("seqs", [[(9, 20), (40, 41)], [(1, 64)]])
def test_append_to_a_pool_with_k_and_v_beside_each_other_in_a_row(monkeypatch, seqs):
    """[pages, page_size, 2, kv_heads, head_dim]"""
    plain = cu.build

    def build(*args, **kw):
        cache, table, lens = plain(*args, **kw)
        both = torch.stack([cache.k, cache.v]).permute(1, 3, 0, 2, 4).contiguous()
        return Cache(*(both[:, :, i].transpose(1, 2) for i in (0, 1))), table, lens

    monkeypatch.setattr(cu, "build", build)
    cache, table, lens = check(seqs, BF16, BF16, 4, 2, 72, 32)
    assert cache.k.stride() == (32 * 2 * 2 * 72, 72, 2 * 2 * 72, 1)
    q = torch.randn(len(seqs), 4, 72, device="cuda").to(BF16)
    out, _ = cache_attention(q, cache, table, lens)
    want, _ = cu.attention(q, cache, table, [s[1] for s in seqs], list(range(len(seqs) + 1)))
    bu.assert_within(out, want["out"], want["out_bound"], "out")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale,maximum", [(1.0, None), (0.37, None), (0.1, 0.0087890625), (0.05, 0.00439453125)])
def test_every_maximum_gets_the_group_scale_that_the_header_states(scale, maximum, dtype):
    """max|y| times the binary32 value of 1 / (6 v_scale), rounded to binary32 and then to e4m3: for a few maxima and
    scales the neighbour of the quotient's."""
    top = torch.arange(0x7C00 if dtype == F16 else 0x7F80, dtype=torch.int16, device="cuda").view(dtype)
    rows = top.numel() // 8
    y = torch.zeros(rows, 8, 16, dtype=dtype, device="cuda")
    y[:, :, 5] = -top.view(rows, 8)
    cache = Cache.empty(rows // 256 + 1, 1, 128, page_size=256, dtype="e2m1", v_scale=scale)
    table = torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None]
    w = torch.ones(128, device="cuda")
    qkv = torch.zeros(rows, 3 * 128, dtype=dtype, device="cuda")
    qkv[:, 256:] = y.view(rows, 128)
    cache_append(qkv, w, w, cache, table, torch.tensor([rows], dtype=torch.int32, device="cuda"), heads=1, rotary_dim=0)
    got = cache.v_scales.view(torch.uint8).view(-1, 8)[:rows].flatten()
    held = float(torch.tensor(scale))  # what binary32 holds of it

    def e4m3(x):
        return x.float().clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)

    r = torch.tensor(1.0 / (6.0 * held), dtype=torch.float64, device="cuda").float()
    assert torch.equal(got, e4m3(top.float() * r))
    if maximum:  # the quotient is just below the middle of codes 7 and 8, the product on it
        assert maximum / (6.0 * held) < 7.5 * 2.0 ** -9 and got[top == maximum].tolist() == [8]


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("exponent", [0, 20, 28, 36, 40])
def test_channels_far_below_a_rows_largest_over_4_bits(exponent, rows):
    """bfloat16 rows with one channel of 2^exponent, which meets zeros: the others are kept to 2^-39 of it."""
    lens = [300, 200]
    cache, table, kv_lens = cu.build(lens, 1, 64, 64, "e2m1", v_scale=0.5)
    cache.k[..., 3] &= 0xF0  # channel 6 of every key: code 0
    q = torch.randn(2 * rows, 4, 64, device="cuda").to(BF16)
    q[..., 6] = 2.0 ** exponent
    out, lse = cache_attention(q, cache, table, kv_lens)
    want, _ = cu.attention(q, cache, table, lens, [0, rows, 2 * rows])
    k = torch.nan_to_num(cu.values(cache)[0], nan=0.0).abs().sum(-1).amax()
    off = 2.0 ** -39 * 2.0 ** exponent * float(k) / 8  # of a score, in binary64
    bu.assert_within(lse.t(), want["lse"], want["lse_bound"] + off, "lse")
    if off < 2.0 ** -8:  # scores and lse off by e each move a weight by a factor of exp(2 e), below 1 + 2.01 e
        spread = 2.01 * off * torch.nan_to_num(cu.values(cache)[1], nan=0.0).abs().amax()
        bu.assert_within(out, want["out"], want["out_bound"] + spread, "out")
