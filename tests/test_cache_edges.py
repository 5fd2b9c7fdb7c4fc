"""The paged cache's operators, without a GPU, where one call could spoil the
next or a value or layout lies at the edge of what is allowed."""
import copy
import math
import random

import pytest

torch = pytest.importorskip("torch")

import test_cache_checks as checks  # noqa: E402
from test_cache_checks import no_gpu  # noqa: E402, F401
from video_vae_decoder_qkv_gb300 import Cache, attention, block, cache as cache_module, cache_attention, h3qk  # noqa: E402

F16, I32 = torch.float16, torch.int32


@pytest.fixture
def packed_calls(monkeypatch):
    """Calls of the binding go into a list, and no further."""
    passed = []
    monkeypatch.setattr(block, "_sizes", {})
    monkeypatch.setattr(block, "_call", lambda name, dev, *args: passed.append(args))
    monkeypatch.setattr(block, "_stream", lambda dev: None)
    monkeypatch.setattr(cache_module, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    return passed


BAD_BENDS = [dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf), dict(softcap=1e-50), dict(softcap=1e39),
             dict(scale=math.inf), dict(scale=math.nan), dict(scale=-1.0), dict(scale=0.0), dict(scale=1e-50),
             dict(scale=1e39)]


@pytest.mark.parametrize("bad", BAD_BENDS, ids=str)
def test_a_refused_call_leaves_the_next_ones_workspace(packed_calls, bad):
    """Refused before a size is kept for it: calls of the same sizes get the workspace that the library asks for."""
    cache = Cache.empty(64, 8, 128, device="cpu", dtype=F16)
    table, lens = torch.zeros(4, 256, dtype=I32), torch.ones(4, dtype=I32)
    for rows in (4, 400):
        q = torch.empty(rows, 40, 128, dtype=F16)
        with pytest.raises(ValueError):
            cache_attention(q, cache, table, lens, **bad)
        assert not packed_calls
        for good in (dict(), dict(softcap=3.0), dict(scale=0.5)):
            cache_attention(q, cache, table, lens, **good)
            pool, call, _ = packed_calls.pop()
            want = block._fn("h3qk_cache_attention_workspace_bytes")(pool, call)
            assert want > 0 and cache_module._ATTN.unpack(call)[-1] == want


@pytest.mark.parametrize("bad", BAD_BENDS, ids=str)
def test_a_refused_call_leaves_the_next_ones_workspace_dense(packed_calls, bad):
    q, k = torch.empty(1, 16, 1, 64, dtype=F16), torch.empty(1, 16, 4896, 64, dtype=F16)
    with pytest.raises(ValueError):
        attention(q, k, k, **bad)
    attention(q, k, k)
    packed, _ = packed_calls.pop()
    want = block._fn("h3qk_attention_workspace_bytes")(packed)
    assert want > 0 and block._ATTN.unpack(packed)[28] == want


@pytest.mark.parametrize("scale", [1e-50, 2.0 ** -118, 2.0 ** 118, 1e39, -1.0])
def test_tensor_scales_that_the_rounding_cannot_take_are_refused(scale):
    for name in ("k_scale", "v_scale"):
        with pytest.raises(ValueError, match=name):
            Cache(*checks.codes(), **{name: scale})
        with pytest.raises(ValueError, match=name):
            Cache.empty(4, 2, 64, dtype="e2m1", device="cpu", **{name: scale})


@pytest.mark.parametrize("scale,want", [(2.0 ** -149, h3qk.ERR_INVALID_ARG), (2.0 ** -118, h3qk.ERR_INVALID_ARG),
                                        (2.0 ** 118, h3qk.ERR_INVALID_ARG), (2.0 ** -117, h3qk.ERR_CUDA),
                                        (2.0 ** 117, h3qk.ERR_CUDA), (0.0, h3qk.ERR_CUDA)])
def test_tensor_scales_of_the_library(no_gpu, scale, want):  # noqa: F811
    for name in ("k_scale", "v_scale"):
        kw = {**checks.E2M1, name: scale}
        assert checks.c_append(**kw) == want and checks.c_attend(**kw) == want and checks.c_read(**kw) == want


A = checks.A
BOTH_IN_A_ROW = dict(v=A + 256, k_st=(8192, 64, 256), v_st=(8192, 64, 256))  # [pages, page_size, 2, kv_heads, head_dim]
CODES_IN_A_PAGE = dict(checks.E2M1, v=A + 1024, k_st=(4096, 2048, 32), v_st=(4096, 2048, 32))  # [pages, kv_heads, 2, ...]
ALL_OF_A_HEAD = dict(checks.E2M1, v=A + 1024, ks=A + 2048, vs=A + 2176, k_st=(4608, 2304, 32), v_st=(4608, 2304, 32),
                     ks_st=(4608, 2304, 4), vs_st=(4608, 2304, 4))


@pytest.mark.parametrize("kw,want", [
    (BOTH_IN_A_ROW, h3qk.ERR_CUDA), ({**BOTH_IN_A_ROW, "v": A + 128}, h3qk.ERR_ALIAS),
    ({**BOTH_IN_A_ROW, "v": A + 384}, h3qk.ERR_ALIAS), ({**BOTH_IN_A_ROW, "pages": 1}, h3qk.ERR_CUDA),
    ({**BOTH_IN_A_ROW, "v": A - 256}, h3qk.ERR_CUDA), ({**BOTH_IN_A_ROW, "v": A + 512 + 256}, h3qk.ERR_CUDA),
    ({**BOTH_IN_A_ROW, "v": A + 512}, h3qk.ERR_ALIAS), ({**BOTH_IN_A_ROW, "v_st": (8192, 64, 128)}, h3qk.ERR_ALIAS),
    (CODES_IN_A_PAGE, h3qk.ERR_CUDA), ({**CODES_IN_A_PAGE, "v": A + 512}, h3qk.ERR_ALIAS),
    (ALL_OF_A_HEAD, h3qk.ERR_CUDA), ({**ALL_OF_A_HEAD, "ks": A + 2048 - 16}, h3qk.ERR_ALIAS),
    ({**ALL_OF_A_HEAD, "vs": A + 2176 + 16}, h3qk.ERR_ALIAS),
])
def test_pools_whose_parts_lie_between_one_another(no_gpu, kw, want):  # noqa: F811
    assert checks.c_append(**kw) == want
    assert checks.c_attend(**kw) == h3qk.ERR_CUDA  # (reading may overlap as it likes)


def test_no_overlap_of_a_written_pool_is_missed(no_gpu):  # noqa: F811
    """Small pools of random strides, against the bytes that their rows have, counted one by one."""
    rng = random.Random(1)
    taken = 0
    for _ in range(3000):
        kv, pages, page = rng.choice((1, 2, 3)), rng.choice((1, 2, 3)), 16
        def strides():
            order, step, got = [("head", kv), ("row", page), ("item", pages)], 8, {}
            rng.shuffle(order)
            for name, n in order:
                got[name] = step * rng.choice((1, 1, 2, 3))
                step = got[name] * n
            return got["item"], got["head"], got["row"]

        k_st = strides()
        v_st = k_st if rng.random() < 0.7 else strides()
        apart = 16 * rng.randrange(-60, 60)
        every = []
        for st in (k_st, v_st):
            every.append([2 * (p * st[0] + h * st[1] + r * st[2]) for p in range(pages) for h in range(kv) for r in range(page)])
        k, v = ({at // 16 + off for at in rows} for rows, off in zip(every, (0, apart // 16)))
        apart_rows = len(k) == len(every[0]) and len(v) == len(every[1]) and not k & v
        got = checks.c_append(dict(heads=kv, rotary=0), kv_heads=kv, pages=pages, page_size=page, head_dim=8, k_st=k_st,
                              v_st=v_st, v=A + apart)
        assert got in (h3qk.ERR_ALIAS, h3qk.ERR_CUDA)
        if got == h3qk.ERR_CUDA:
            assert apart_rows, (kv, pages, k_st, v_st, apart)
            taken += 1
        elif k_st == v_st:
            assert not apart_rows, (kv, pages, k_st, v_st, apart)
    assert taken > 300


def called(packed_calls, cache):
    """h3qk_cache of a call, unpacked."""
    cache_attention(torch.empty(2, 4, 64, dtype=F16), cache, torch.zeros(2, 4, dtype=I32), torch.ones(2, dtype=I32))
    pool = packed_calls.pop()[0]
    return cache_module._POOL.unpack(pool[:cache_module._POOL.size])


CHANGES = {
    "shape": lambda t: t.resize_(2, 2, 64, 64), "fewer": lambda t: t.resize_(1, 2, 64, 64), "more": lambda t: t.resize_(300, 2, 64, 64),
    "turned": lambda t: t.transpose_(1, 2), "set": lambda t: t.set_(torch.empty(1, 2, 64, 64, dtype=t.dtype)),
    "data": lambda t: setattr(t, "data", torch.empty(1, 2, 64, 64, dtype=t.dtype)),
    "part": lambda t: t.set_(t.untyped_storage(), 8, (1, 2, 64, 56)),
}


@pytest.mark.parametrize("change", list(CHANGES))
@pytest.mark.parametrize("fmt", ["e2m1", F16])
def test_tensors_that_are_changed_in_place(packed_calls, fmt, change):
    """Other memory is refused; other shapes of the same memory leave the cache as it was made, within that memory."""
    for name in ("k", "v") if fmt == F16 else ("k", "v", "k_scales", "v_scales"):
        cache = Cache.empty(9, 2, 64, device="cpu", dtype=fmt)
        was = called(packed_calls, cache)
        t = getattr(cache, name)
        CHANGES[change](t)
        moved = t.data_ptr() != was[5 + ("k", "v", "k_scales", "v_scales").index(name)]
        assert moved or change not in ("set", "data", "part", "more")
        if moved:
            with pytest.raises(ValueError, match="other memory"):
                called(packed_calls, cache)
            assert not packed_calls
            continue
        assert called(packed_calls, cache) == was
        assert t.untyped_storage().nbytes() >= 9 * 2 * 64 * (4 if "scales" in name else 32)


@pytest.mark.parametrize("fmt", ["e2m1", F16])
def test_copies_of_a_cache_can_be_called(packed_calls, fmt):
    cache = Cache.empty(9, 2, 64, device="cpu", dtype=fmt)
    was = called(packed_calls, cache)
    assert called(packed_calls, copy.copy(cache)) == was
    other = copy.deepcopy(cache)
    now = called(packed_calls, other)
    assert now[:5] == was[:5] and now[9:] == was[9:] and now[5] == other.k.data_ptr() != was[5]


def test_the_memory_of_a_cache_stays_its_own(packed_calls):
    """A tensor that lost its memory and is given a smaller one: that cannot lie at the old address."""
    cache = Cache.empty(64, 2, 64, device="cpu", dtype=F16)
    for _ in range(20):
        cache.k.set_()
        cache.k.set_(torch.empty(1, 2, 64, 64, dtype=F16))
        with pytest.raises(ValueError, match="other memory"):
            called(packed_calls, cache)


@pytest.mark.parametrize("tokens,max_rows,want", [
    (2 ** 30 - 1, 0, h3qk.ERR_INVALID_ARG), (2 ** 30 - 127, 0, h3qk.ERR_INVALID_ARG), (2 ** 30 - 128, 0, h3qk.ERR_CUDA),
    (2 ** 30 - 1, 2 ** 30 - 128, h3qk.ERR_CUDA), (2 ** 30 - 1, 1, h3qk.ERR_CUDA),
])
def test_rows_of_a_sequence_fit_31_bits_to_full_tiles(no_gpu, tokens, max_rows, want):  # noqa: F811
    """The kernel counts a sequence's rows times the heads of a K/V head, rounded up to tiles of 256, in 31 bits."""
    call = dict(tokens=tokens, max_rows=max_rows, heads=2, q=1 << 44, out=1 << 45, lse=1 << 46, qt=128, ot=128,
                offsets=1 << 47)
    assert checks.c_attend(call, kv_heads=1) == want
