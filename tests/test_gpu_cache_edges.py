"""The paged cache's operators where their documentation allows more than
ordinary calls make: rows that are not finite beside rows that are."""
import math

import block_util as bu
import cache_util as cu
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from video_vae_decoder_qkv_gb300 import cache_attention  # noqa: E402

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
