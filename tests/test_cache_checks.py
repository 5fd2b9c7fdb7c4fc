"""Refusals of the paged cache's operators, without a GPU: the binding on meta
tensors, and the C-ABI on fake addresses that every call rejects before it
would touch them."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from video_vae_decoder_qkv_gb300 import (Cache, block, cache as cache_module, cache_append, cache_attention,  # noqa: E402
                                         cache_read, h3qk)

M = torch.device("meta")
F16, BF16, F32, I32, U8, E4M3 = (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.uint8,
                                 torch.float8_e4m3fn)
A = 0x10000000
INVALID, MISALIGNED, ALIAS = h3qk.ERR_INVALID_ARG, h3qk.ERR_MISALIGNED, h3qk.ERR_ALIAS


def t(*shape, dtype=F16):
    return torch.empty(shape, dtype=dtype, device=M)


@pytest.fixture
def no_gpu():
    """Fake addresses must never reach a kernel: only where no GPU exists."""
    if torch.cuda.is_available():
        pytest.skip("fake-address checks run only on hosts without a GPU")


def codes(dim=64, page=32, heads=2, scales=True):
    k = t(9, heads, page, dim // 2, dtype=U8)
    s = t(9, heads, page, dim // 16, dtype=E4M3) if scales else None
    return k, k, s, s


@pytest.mark.parametrize("args,kw,error", [
    ((t(9, 2, 32, 64, dtype=F32), t(9, 2, 32, 64, dtype=F32)), {}, TypeError),
    ((t(9, 2, 64), t(9, 2, 64)), {}, ValueError),
    ((t(9, 2, 24, 64), t(9, 2, 24, 64)), {}, ValueError),
    ((t(9, 2, 8, 64), t(9, 2, 8, 64)), {}, ValueError),
    ((t(9, 2, 32, 60), t(9, 2, 32, 60)), {}, ValueError),
    ((t(9, 2, 32, 136), t(9, 2, 32, 136)), {}, ValueError),
    ((t(9, 0, 32, 64), t(9, 0, 32, 64)), {}, ValueError),
    ((t(9, 2, 32, 64), t(9, 2, 32, 72)), {}, ValueError),
    ((t(9, 2, 32, 64), t(9, 2, 32, 64, dtype=BF16)), {}, TypeError),
    ((t(9, 2, 64, 32).transpose(2, 3), t(9, 2, 32, 64)), {}, ValueError),
    ((t(9, 2, 32, 64), t(9, 2, 32, 64), t(9, 2, 32, 4, dtype=E4M3), t(9, 2, 32, 4, dtype=E4M3)), {}, ValueError),
    ((t(9, 2, 32, 64), t(9, 2, 32, 64)), dict(k_scale=2.0), ValueError),
    (codes(scales=False), {}, ValueError),
    (codes(dim=48), {}, ValueError),
    (codes(), dict(v_scale=0.0), ValueError),
    (codes(), dict(k_scale=math.inf), ValueError),
    (codes(), dict(k_scale=math.nan), ValueError),
    ((*codes()[:2], t(9, 2, 32, 4, dtype=U8), t(9, 2, 32, 4, dtype=U8)), {}, TypeError),
    ((*codes()[:2], t(9, 2, 32, 2, dtype=E4M3), t(9, 2, 32, 4, dtype=E4M3)), {}, ValueError),
])
def test_cache_refuses(args, kw, error):
    with pytest.raises(error):
        Cache(*args, **kw)


def test_cache_empty_refuses_and_describes():
    with pytest.raises(ValueError):
        Cache.empty(4, 2, 48, dtype="e2m1", device="cpu")
    c = Cache.empty(4, 2, 96, dtype="e2m1", page_size=16, device="cpu")
    assert c.k.shape == (4, 2, 16, 48) and c.v_scales.shape == (4, 2, 16, 6) and c.head_dim == 96 and c.dtype == "e2m1"
    c = Cache.empty(4, 2, 40, dtype=F16, device="cpu")
    assert c.k.shape == (4, 2, 64, 40) and c.k_scales is None and c.dtype == F16


CACHE = Cache(t(9, 2, 32, 64), t(9, 2, 32, 64))
CODES = Cache(*codes())
TABLE, LENS = t(3, 4, dtype=I32), t(3, dtype=I32)
POOL_ERRORS = [
    (dict(table=t(3, 4, dtype=torch.int64)), TypeError), (dict(table=t(12, dtype=I32)), ValueError),
    (dict(table=t(4, 3, dtype=I32).t()), ValueError), (dict(table=t(1, 4, dtype=I32).expand(3, 4)), ValueError),
    (dict(table=t(3, 1 << 25, dtype=I32)), ValueError), (dict(table=t(0, 4, dtype=I32), lens=t(0, dtype=I32)), ValueError),
    (dict(table=torch.empty(3, 4, dtype=I32)), ValueError), (dict(lens=None), ValueError),
    (dict(lens=t(4, dtype=I32)), ValueError), (dict(lens=t(3, dtype=torch.int64)), TypeError),
    (dict(lens=t(6, dtype=I32)[::2]), ValueError),
]


def append(**kw):
    a = dict(qkv=t(6, 8 * 64), wq=t(64, dtype=F32), wk=t(64, dtype=F32), cache=CACHE, table=TABLE, lens=LENS)
    more = dict(heads=4, rotary_dim=64)
    more.update({k: v for k, v in kw.items() if k not in a})
    a.update({k: v for k, v in kw.items() if k in a})
    return cache_append(*a.values(), **more)


@pytest.mark.parametrize("kw,error", POOL_ERRORS + [
    (dict(qkv=t(6, 512, dtype=F32)), TypeError), (dict(qkv=t(6, 512, dtype=BF16)), TypeError),
    (dict(qkv=t(6, 511)), ValueError), (dict(qkv=t(512, 6).t()), ValueError), (dict(qkv=t(1, 512).expand(6, 512)), ValueError),
    (dict(qkv=t(5, 512)), ValueError), (dict(heads=0), ValueError), (dict(heads=5), ValueError),
    (dict(wq=t(32, dtype=F32)), ValueError), (dict(wk=t(64)), TypeError), (dict(positions=t(5, 3, dtype=I32)), ValueError),
    (dict(positions=t(6, 3)), TypeError), (dict(n_axes=3), ValueError), (dict(q_offsets=t(3, dtype=I32)), ValueError),
    (dict(q_offsets=t(4, dtype=torch.int64)), TypeError), (dict(out=t(6, 4, 32)), ValueError),
    (dict(out=t(6, 4, 64, dtype=BF16)), TypeError),
])
def test_append_refuses(kw, error):
    with pytest.raises(error):
        append(**kw)


def attend(**kw):
    a = dict(q=t(6, 4, 64), cache=CACHE, table=TABLE, lens=LENS)
    more = {k: v for k, v in kw.items() if k not in a}
    a.update({k: v for k, v in kw.items() if k in a})
    return cache_attention(*a.values(), **more)


@pytest.mark.parametrize("kw,error", POOL_ERRORS + [
    (dict(q=t(6, 4, 64, dtype=F32)), TypeError), (dict(q=t(6, 4, 64, dtype=BF16)), TypeError), (dict(q=t(6, 256)), ValueError),
    (dict(q=t(6, 3, 64)), ValueError), (dict(q=t(6, 4, 32)), ValueError), (dict(q=t(6, 64, 4).transpose(1, 2)), ValueError),
    (dict(q=t(5, 4, 64)), ValueError), (dict(scale=0.0), ValueError), (dict(scale=math.nan), ValueError),
    (dict(max_rows=0), ValueError), (dict(causal=False, prefix_lens=t(3, dtype=I32)), ValueError),
    (dict(prefix_lens=t(2, dtype=I32)), ValueError), (dict(q_offsets=t(3, dtype=I32)), ValueError),
    (dict(slopes=t(2, dtype=F32)), ValueError), (dict(slopes=t(4)), TypeError), (dict(out=t(6, 4, 32)), ValueError),
    (dict(out=t(6, 4, 64, dtype=BF16)), TypeError), (dict(lse=t(4, 5, dtype=F32)), ValueError), (dict(lse=t(4, 6)), TypeError),
])
def test_attention_refuses(kw, error):
    with pytest.raises(error):
        attend(**kw)


@pytest.mark.parametrize("kw,error", [
    (dict(dtype=BF16), TypeError), (dict(dtype=F32), TypeError), (dict(rows=-1), ValueError), (dict(rows=1 << 30), ValueError),
    (dict(starts=t(2, dtype=I32)), ValueError), (dict(out_k=t(3, 2, 5, 64), rows=4), ValueError),
    (dict(out_v=t(3, 2, 4, 64, dtype=BF16), rows=4), TypeError),
])
def test_read_refuses(kw, error):
    with pytest.raises(error):
        cache_read(CACHE, TABLE, LENS, **kw)


def test_operators_refuse_host_tensors():
    c = Cache.empty(4, 2, 64, device="cpu", dtype=F16)
    table, lens = torch.zeros(1, 2, dtype=I32), torch.ones(1, dtype=I32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        cache_attention(torch.zeros(1, 4, 64, dtype=F16), c, table, lens)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        cache_read(c, table, lens)


# ---- the C-ABI --------------------------------------------------------------------------------------------------------
POOL = dict(format=h3qk.FP16, kv_heads=2, head_dim=64, page_size=32, pages=9, k=A, v=A + 0x1000000, ks=0, vs=0,
            k_st=(4096, 2048, 64), v_st=(4096, 2048, 64), ks_st=(0, 0, 0), vs_st=(0, 0, 0), k_scale=1.0, v_scale=1.0,
            batch=3, max_pages=4, table=A + 0x2000000, table_stride=0, lens=A + 0x2001000)
E2M1 = dict(format=cache_module.E2M1, ks=A + 0x3000000, vs=A + 0x3100000, k_st=(2048, 1024, 32), v_st=(2048, 1024, 32),
            ks_st=(256, 128, 4), vs_st=(256, 128, 4))


def pool(**kw):
    a = {**POOL, **kw}
    return cache_module._POOL.pack(*(a[n] for n in ("format", "kv_heads", "head_dim", "page_size", "pages", "k", "v", "ks", "vs")),
                                   *a["k_st"], *a["v_st"], *a["ks_st"], *a["vs_st"], a["k_scale"], a["v_scale"]) + \
        cache_module._TABLE.pack(*(a[n] for n in ("batch", "max_pages", "table", "table_stride", "lens")))


def c_attend(call=None, **kw):
    a = dict(dtype=h3qk.FP16, heads=4, causal=1, max_rows=0, scale=0.0, softcap=0.0, tokens=6, q=A + 0x4000000,
             out=A + 0x5000000, qt=256, qh=64, ot=256, oh=64, lse=A + 0x6000000, slopes=0, prefix=0, offsets=0,
             ws=A + 0x7000000, ws_bytes=1 << 27)
    a.update(call or {})
    return block._fn("h3qk_cache_attention")(pool(**kw), cache_module._ATTN.pack(*a.values()), None)


BAD_POOLS = [
    (dict(format=h3qk.E4M3), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=65536), INVALID), (dict(batch=0), INVALID),
    (dict(head_dim=60), INVALID), (dict(head_dim=136), INVALID), (dict(page_size=24), INVALID), (dict(page_size=8), INVALID),
    (dict(pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(max_pages=1 << 25), INVALID),
    (dict(table_stride=3), INVALID), (dict(lens=0), INVALID), (dict(table=0), INVALID), (dict(lens=A + 2), MISALIGNED),
    (dict(table=A + 0x2000002), MISALIGNED), (dict(k_scale=2.0), INVALID), (dict(k_scale=-1.0), INVALID),
    (dict(v_scale=math.nan), INVALID), (dict(ks=A), INVALID), (dict(k=0), INVALID), (dict(k=A + 8), MISALIGNED),
    (dict(k_st=(4096, 2048, 60)), INVALID), (dict(k_st=(4096, 2048, 68)), MISALIGNED), (dict(v_st=(4097, 2048, 64)), MISALIGNED),
    (dict(v_st=(-4096, 2048, 64)), INVALID), (dict(v_st=(1 << 36, 2048, 64)), INVALID),
    ({**E2M1, "head_dim": 48}, INVALID), ({**E2M1, "ks": 0}, INVALID), ({**E2M1, "vs": A + 0x3100008}, MISALIGNED),
    ({**E2M1, "k_st": (2048, 1024, 40)}, INVALID), ({**E2M1, "k_st": (2040, 1024, 32)}, MISALIGNED),
    ({**E2M1, "ks_st": (256, 128, 8)}, INVALID), ({**E2M1, "k_scale": math.inf}, INVALID),
]


@pytest.mark.parametrize("kw,want", BAD_POOLS)
def test_pools_are_checked(no_gpu, kw, want):
    assert c_attend(**kw) == want
    assert c_append(**kw) == want
    assert c_read(**kw) == want


@pytest.mark.parametrize("call,want", [
    (dict(dtype=block.FP32), INVALID), (dict(dtype=h3qk.BF16), INVALID), (dict(heads=3), INVALID), (dict(heads=0), INVALID),
    (dict(causal=2), INVALID), (dict(max_rows=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(softcap=math.nan), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=5), INVALID), (dict(tokens=1 << 30), INVALID),
    (dict(tokens=900000000, heads=4), INVALID), (dict(causal=0, prefix=A), INVALID), (dict(q=0), INVALID), (dict(out=0), INVALID),
    (dict(lse=0), INVALID), (dict(qh=56), INVALID), (dict(qt=-256), INVALID), (dict(qh=68), MISALIGNED),
    (dict(q=A + 0x4000008), MISALIGNED), (dict(lse=A + 0x6000002), MISALIGNED), (dict(offsets=A + 0x8000002), MISALIGNED),
    (dict(ot=128), ALIAS), (dict(out=A + 0x4000000), ALIAS), (dict(out=A), ALIAS), (dict(lse=A + 0x2001000), ALIAS),
    (dict(lse=A + 0x5000000), ALIAS), (dict(tokens=60, ws=0), INVALID), (dict(tokens=60, ws_bytes=64), INVALID),
    (dict(tokens=60, ws=A + 0x7000008), MISALIGNED), (dict(tokens=60, ws=A), ALIAS),
    (dict(), h3qk.ERR_CUDA), (dict(ws=0, ws_bytes=0), h3qk.ERR_CUDA), (dict(tokens=0, q=0, out=0, lse=0), h3qk.OK),
])
def test_attention_calls_are_checked(no_gpu, call, want):
    assert c_attend(call) == want


def c_append(call=None, opts=None, **kw):
    o = h3qk.default_opts()
    o.in_dtype, o.n_axes = h3qk.FP16, 1
    for n, v in (opts or {}).items():
        setattr(o, n, v)
    a = dict(qkv=A + 0x4000000, wq=A + 0x5000000, wk=A + 0x5001000, pos=0, tokens=6, heads=4, rotary=64, offsets=0,
             out=A + 0x6000000)
    a.update(call or {})
    return block._fn("h3qk_cache_append")(pool(**kw), *a.values(), ctypes.byref(o), None)


@pytest.mark.parametrize("call,opts,want", [
    (dict(heads=0), {}, INVALID), (dict(tokens=-1), {}, INVALID), (dict(tokens=5), {}, INVALID), (dict(rotary=63), {}, INVALID),
    (dict(rotary=66), {}, INVALID), (dict(qkv=0), {}, INVALID), (dict(wq=0), {}, INVALID), (dict(out=0), {}, INVALID),
    (dict(), dict(in_dtype=h3qk.BF16), INVALID), (dict(), dict(n_axes=3), INVALID), (dict(), dict(qkv_row_stride=504), INVALID),
    (dict(), dict(qkv_row_stride=516), MISALIGNED), (dict(), dict(eps=-1.0), INVALID), (dict(qkv=A + 0x4000004), {}, MISALIGNED),
    (dict(out=A + 0x6000008), {}, MISALIGNED), (dict(offsets=A + 2), {}, MISALIGNED), (dict(out=A + 0x4000000), {}, ALIAS),
    (dict(out=A), {}, ALIAS), (dict(out=A + 0x5000000), {}, ALIAS), (dict(out=A + 0x2000000), {}, ALIAS),
    (dict(qkv=A + 0x1000000), {}, ALIAS), (dict(offsets=A), {}, ALIAS), (dict(), {}, h3qk.ERR_CUDA),
    (dict(pos=A + 0x8000000), dict(n_axes=3, axis_dims=(ctypes.c_int32 * 3)(32, 16, 16)), h3qk.ERR_CUDA),
    (dict(tokens=0, qkv=0, out=0), {}, h3qk.OK),
])
def test_append_calls_are_checked(no_gpu, call, opts, want):
    assert c_append(call, opts) == want


@pytest.mark.parametrize("kw,want", [
    (dict(v=A), ALIAS), (dict(v=A + 2048), ALIAS), (dict(k_st=(2048, 2048, 64)), ALIAS), (dict(k_st=(4096, 1024, 64)), ALIAS),
    # K and V of a page beside each other
    (dict(v=A + 8192, k_st=(8192, 2048, 64), v_st=(8192, 2048, 64)), h3qk.ERR_CUDA),
    (dict(v=A + 4096, k_st=(8192, 2048, 64), v_st=(8192, 2048, 64)), ALIAS),
    # heads beside each other in a row
    (dict(k_st=(4096, 64, 128), v_st=(4096, 64, 128)), h3qk.ERR_CUDA),
    ({**E2M1, "vs": A + 0x3000000}, ALIAS), ({**E2M1, "ks": A}, ALIAS), (E2M1, h3qk.ERR_CUDA),
])
def test_written_pools_do_not_overlap(no_gpu, kw, want):
    assert c_append(**kw) == want


def c_read(call=None, **kw):
    a = dict(starts=0, rows=10, dtype=h3qk.FP16, k=A + 0x4000000, v=A + 0x5000000)
    a.update(call or {})
    return block._fn("h3qk_cache_read")(pool(**kw), *a.values(), None)


@pytest.mark.parametrize("call,want", [
    (dict(rows=-1), INVALID), (dict(dtype=h3qk.BF16), INVALID), (dict(dtype=block.FP32), INVALID), (dict(k=0), INVALID),
    (dict(v=A + 0x5000008), MISALIGNED), (dict(starts=A + 2), MISALIGNED), (dict(v=A + 0x4000000), ALIAS), (dict(k=A), ALIAS),
    (dict(k=A + 0x2001000), ALIAS), (dict(), h3qk.ERR_CUDA), (dict(rows=0, k=0, v=0), h3qk.OK),
])
def test_read_calls_are_checked(no_gpu, call, want):
    assert c_read(call) == want


def test_null_calls(no_gpu):
    assert block._fn("h3qk_cache_attention")(None, None, None) == INVALID
    assert block._fn("h3qk_cache_attention")(pool(), None, None) == INVALID
    assert block._fn("h3qk_cache_attention_workspace_bytes")(None, None) == 0
    assert block._fn("h3qk_cache_read")(None, None, 1, 1, None, None, None) == INVALID


def test_structs_are_packed_as_the_header_lays_them_out():
    assert len(pool()) == 192 and cache_module._ATTN.size == 128


@pytest.mark.parametrize("name", ["k", "v", "k_scales", "k_scale", "v_scale", "pages", "dtype"])
def test_a_cache_stays_what_it_was_made_of(name):
    c = Cache(*codes())
    was = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, was)
    assert getattr(c, name) is was
