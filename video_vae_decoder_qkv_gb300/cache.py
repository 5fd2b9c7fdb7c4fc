"""Python binding of the paged cache: appending prepared keys and values,
attention over the cache, and reading rows back.

As in ``block``, this only checks tensors and passes their addresses: each
operator runs in the library's CUDA kernels on the current stream, or on the
one passed as ``stream``, and workspaces come from torch's allocator unless
the caller passes one.  These are operators of serving; they carry no
autograd graph.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import block, h3qk
from .block import _DTYPES, _need_bend, _need_lens, _on_stream, _stream, _workspace
from .h3qk import _need, _ptr

E2M1 = 5
_P, _I32, _I64, _SZ, _INT = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
block._SIGNATURES.update({
    "h3qk_cache_append": (_INT, [ctypes.c_char_p, _P, _P, _P, _P, _I64, _I32, _I32, _P, _P, ctypes.POINTER(h3qk.Opts), _P]),
    "h3qk_cache_attention_workspace_bytes": (_SZ, [ctypes.c_char_p, ctypes.c_char_p]),
    "h3qk_cache_attention": (_INT, [ctypes.c_char_p, ctypes.c_char_p, _P]),
    "h3qk_cache_read": (_INT, [ctypes.c_char_p, _P, _I64, _INT, _P, _P, _P]),
})

# h3qk_cache and h3qk_cache_attn (include/h3qk.h), each packed in one step
_POOL = struct.Struct("@4iq4P12q2f")
_POINTERS = struct.Struct("@4P")  # _POOL's, which begin at byte 24
_TABLE = struct.Struct("@2iPqP")
_ATTN = struct.Struct("@4i2fq2P4q5PN")


class Cache:
    """Keys and values in pages (h3qk_cache).

    16 bits: ``k`` and ``v`` are float16 or bfloat16 [pages, kv_heads,
    page_size, head_dim], head_dim a multiple of 8 up to 128; any page, head
    and row strides that are multiples of 8 elements will do, so a pool laid
    out [pages, page_size, kv_heads, head_dim] is passed as its ``transpose(1,
    2)``.  4 bits: ``k`` and ``v`` are uint8 codes [pages, kv_heads,
    page_size, head_dim / 2] and ``k_scales``, ``v_scales`` float8_e4m3fn
    [pages, kv_heads, page_size, head_dim / 16], head_dim a multiple of 32 up
    to 128; a value is its e2m1 code (channel 2i in the low half of byte i)
    times its group's scale times ``k_scale`` (``v_scale``; 2^-117 to 2^117).  page_size is a
    power of two from 16 on.  ``Cache.empty`` allocates one.  What a cache is made
    of stays: other tensors or scales are another Cache.  A tensor that is given
    other memory in place (``set_``, ``data``, a ``resize_`` that grows) is
    refused at the next call; one that is only given another shape leaves the
    cache as it was made."""

    __slots__ = ("k", "v", "k_scales", "v_scales", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "head_dim",
                 "dtype", "device", "_held", "_at", "_head", "_tail")

    def __init__(self, k, v, k_scales=None, v_scales=None, *, k_scale: float = 1.0, v_scale: float = 1.0):
        if k.dim() != 4:
            raise ValueError("k and v must be [pages, kv_heads, page_size, head_dim]")
        codes = k.dtype == torch.uint8
        if not codes and k.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"k must be float16, bfloat16 or uint8 codes, got {k.dtype}")
        pages, heads, page, width = k.shape
        dim = 2 * width if codes else width
        step = 32 if codes else 8
        if heads < 1 or dim < step or dim > 128 or dim % step:
            raise ValueError(f"head_dim must be a multiple of {step} up to 128, got {dim}")
        if page < 16 or page > 65536 or page & (page - 1):
            raise ValueError(f"page_size must be a power of two from 16 to 65536, got {page}")
        if codes != (k_scales is not None) or codes != (v_scales is not None):
            raise ValueError("k_scales and v_scales belong to codes, and only to them")
        for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if not 2.0 ** -117 <= s <= 2.0 ** 117:
                raise ValueError(f"{name} must be from 2^-117 to 2^117, got {s}")
            if not codes and s != 1.0:
                raise ValueError(f"{name} belongs to codes")
        strides = []
        for t, name in ((k, "k"), (v, "v")):
            self._need(t, name, (pages, heads, page, width), k.dtype, k.device)
            strides += t.stride()[:3]
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            if t is None:
                strides += (0, 0, 0)
                continue
            self._need(t, name, (pages, heads, page, dim // 16), torch.float8_e4m3fn, k.device)
            strides += t.stride()[:3]
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.dtype, self.device = ("e2m1" if codes else k.dtype), k.device
        # The memory that the strides describe, kept by views of our own: whatever becomes of a tensor in
        # place, nothing else comes to lie at these addresses.
        self._held = tuple(t if t is None else t.detach() for t in (k, v, k_scales, v_scales))
        self._at = _addresses(self)
        # h3qk_cache but for the addresses, which each call takes anew
        packed = _POOL.pack(E2M1 if codes else _DTYPES[k.dtype], heads, dim, page, pages, 0, 0, 0, 0, *strides, self.k_scale,
                            self.v_scale)
        self._head, self._tail = packed[:24], packed[24 + _POINTERS.size:]

    def __setattr__(self, name, value):
        if hasattr(self, "_tail"):
            raise AttributeError(f"{name} of a Cache is fixed: make another Cache")
        object.__setattr__(self, name, value)

    def __reduce__(self):
        """Copies are made of (copies of) the same tensors."""
        return (functools.partial(type(self), k_scale=self.k_scale, v_scale=self.v_scale),
                (self.k, self.v, self.k_scales, self.v_scales))

    @staticmethod
    def _need(t, name, shape, dtype, dev):
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        if t.stride(3) != 1 and shape[3] > 1:
            raise ValueError(f"{name} must have unit stride along head_dim")

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, *, page_size: int = 64, dtype=torch.bfloat16, device="cuda",
              k_scale: float = 1.0, v_scale: float = 1.0):
        """A cache of uninitialised pages; ``dtype`` is a 16-bit type or "e2m1"."""
        if dtype != "e2m1":
            return cls(*(torch.empty((pages, kv_heads, page_size, head_dim), dtype=dtype, device=device) for _ in range(2)),
                       k_scale=k_scale, v_scale=v_scale)
        if head_dim % 32:
            raise ValueError(f"head_dim must be a multiple of 32 up to 128, got {head_dim}")
        codes = (torch.empty((pages, kv_heads, page_size, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2))
        scales = (torch.empty((pages, kv_heads, page_size, head_dim // 16), dtype=torch.uint8, device=device) for _ in range(2))
        return cls(*codes, *(s.view(torch.float8_e4m3fn) for s in scales), k_scale=k_scale, v_scale=v_scale)


def _list(t, name, n, dev):
    """The address of an int32 list of n (0 for none)."""
    if t is None:
        return 0
    if t.dtype is torch.int32 and t.shape == (n,) and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    return _need_lens(t, name, n, dev)  # says what is wrong


def _addresses(cache):
    ks, vs = cache.k_scales, cache.v_scales
    return (cache.k.data_ptr(), cache.v.data_ptr(), 0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr())


def _pool(cache, block_table, kv_lens):
    """h3qk_cache as bytes, after checking the table and the lengths: (packed, batch)."""
    dev = cache.device
    if block_table.dtype is not torch.int32:
        raise TypeError(f"block_table must be torch.int32, got {block_table.dtype}")
    if block_table.dim() != 2 or block_table.device != dev:
        raise ValueError(f"block_table must be [batch, max_pages] on {dev}")
    batch, max_pages = block_table.shape
    across, along = block_table.stride()
    if (along != 1 and max_pages > 1) or (across < max_pages and batch > 1):
        raise ValueError("block_table must have unit stride along a sequence's pages, and no overlapping rows")
    if batch < 1 or max_pages * cache.page_size >= 1 << 30:
        raise ValueError("block_table must hold at least one sequence, and fewer than 2^30 rows of each")
    if kv_lens is None:
        raise ValueError("kv_lens is required")
    at = _addresses(cache)
    if at != cache._at:
        raise ValueError("a tensor of the Cache has other memory than when it was made: make another Cache")
    table = _TABLE.pack(batch, max_pages, block_table.data_ptr(), across if batch > 1 else 0,
                        _list(kv_lens, "kv_lens", batch, dev))
    return cache._head + _POINTERS.pack(*at) + cache._tail + table, batch


def _offsets(q_offsets, batch, tokens, dev):
    if q_offsets is None and tokens % batch:
        raise ValueError(f"{tokens} rows cannot be shared evenly by {batch} sequences: q_offsets is required")
    return _list(q_offsets, "q_offsets", batch + 1, dev)


@functools.lru_cache(maxsize=256)
def _opts(dtype, row_stride, n_axes, axis_dims, theta, eps):
    """h3qk_opts of an append (the library reads it only; filling one takes longer than the call)."""
    o = h3qk.default_opts()
    o.in_dtype = _DTYPES[dtype]
    o.n_axes = n_axes
    if axis_dims is not None:
        o.axis_dims = (ctypes.c_int32 * 3)(*axis_dims, *[0] * (3 - len(axis_dims)))
    o.eps, o.theta, o.batch, o.qkv_row_stride = eps, theta, 1, row_stride
    return ctypes.byref(o)


@_on_stream
def cache_append(qkv, norm_wq, norm_wk, cache, block_table, kv_lens, *, heads: int, rotary_dim: int, positions=None,
                 q_offsets=None, n_axes: int | None = None, axis_dims=None, theta: float = 10000.0, eps: float = 1e-6,
                 out=None):
    """``prepare`` for the new rows of several sequences, with K and V going
    into the cache (h3qk_cache_append).

    qkv: float16 or bfloat16 [tokens, row_stride], each row [Q | K | V] of
    ``heads``, kv_heads and kv_heads head rows (a 16-bit cache's own type).
    ``q_offsets`` (int32 [batch + 1]) says which rows belong to which
    sequence (default: equally many each); ``kv_lens`` (int32 [batch]) are the
    sequences' lengths with the new rows, which become their last ones;
    ``block_table`` (int32 [batch, max_pages]) names each sequence's pages.
    ``positions`` (int32 [tokens, n_axes]) are as for ``prepare``; without
    them a row's place in its sequence is its one position.

    Returns q [tokens, heads, head_dim].  Rows of no sequence leave it and the
    cache as they were; pages that the table does not have, or whose number
    lies outside the pool, are not written."""
    if qkv.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("qkv must be float16 or bfloat16")
    if cache.dtype != "e2m1" and cache.dtype != qkv.dtype:
        raise TypeError(f"qkv must be {cache.dtype} as the cache, got {qkv.dtype}")
    dev, dim = cache.device, cache.head_dim
    if qkv.dim() != 2 or qkv.stride(1) != 1 or qkv.device != dev:
        raise ValueError(f"qkv must be 2-D [tokens, row_stride] with unit inner stride on {dev}")
    tokens, width = qkv.shape
    if heads < 1 or width < (heads + 2 * cache.kv_heads) * dim:
        raise ValueError(f"qkv rows hold {width} values, the call reads {(heads + 2 * cache.kv_heads) * dim}")
    if tokens > 1 and qkv.stride(0) < (heads + 2 * cache.kv_heads) * dim:
        raise ValueError("qkv must not have overlapping rows")
    pool, batch = _pool(cache, block_table, kv_lens)
    offsets = _offsets(q_offsets, batch, tokens, dev)
    if n_axes is None:
        n_axes = 1 if positions is None else positions.shape[1] if positions.dim() == 2 else 3
    if positions is not None:
        _need(positions, "positions", device=dev, dtypes=(torch.int32,), numel=tokens * n_axes)
    elif n_axes != 1 and rotary_dim:
        raise ValueError("positions may be left out for one axis only")
    for w, name in ((norm_wq, "norm_wq"), (norm_wk, "norm_wk")):
        _need(w, name, device=dev, dtypes=(torch.float32,), numel=dim)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=qkv.dtype, device=dev)
    else:
        _need(out, "out", device=dev, dtypes=(qkv.dtype,), numel=tokens * heads * dim)
    o = _opts(qkv.dtype, qkv.stride(0) if tokens > 1 else 0, n_axes, None if axis_dims is None else tuple(axis_dims), theta, eps)
    block._call("h3qk_cache_append", dev, pool, qkv.data_ptr(), norm_wq.data_ptr(), norm_wk.data_ptr(), _ptr(positions),
                tokens, heads, rotary_dim, offsets, out.data_ptr(), o, _stream(dev))
    return out


def _head_rows(t, name, shape, dtype, dev):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return st[0], st[1]


@_on_stream
def cache_attention(q, cache, block_table, kv_lens, *, q_offsets=None, max_rows: int | None = None,
                    scale: float | None = None, softcap: float = 0.0, slopes=None, causal: bool = True, prefix_lens=None,
                    out=None, lse=None, workspace=None):
    """``attention`` with the keys and values of a cache (h3qk_cache_attention).

    q: float16 or bfloat16 [tokens, heads, head_dim] (a 16-bit cache's own
    type; kv_heads divides heads; any token and head strides that are multiples
    of 8 elements), the packed rows of all sequences, with ``q_offsets``,
    ``kv_lens`` and ``block_table`` as for ``cache_append``: a sequence's
    rows are its last ones, and each sees, with ``causal``, the keys up to its
    own and the first ``prefix_lens`` (int32 [batch]); else all of the
    sequence's.  ``max_rows``: no sequence has more rows than that (default:
    q's rows, without q_offsets those of a sequence).  It chooses the kernel,
    which up to 32 packed rows (max_rows times heads per K/V head) is the one for
    few rows: with q_offsets the host does not know the longest sequence, and
    single tokens of a batch take three times as long without it.  The choice
    also goes by the table's width: short ones (8,192 rows) of few sequences
    take one launch, whatever their lengths.
    ``scale``, ``softcap`` and ``slopes`` are ``attention``'s.

    Returns (out, lse): out like q, lse float32 [heads, tokens].  Rows that
    see nothing have out = 0 and lse = -inf; rows of no sequence are left as
    they were (uninitialised without ``out``).  Over 4 bits, bfloat16 rows are
    kept to 2^-39 of their largest magnitude.  The same call gives the same
    bits every time."""
    dtype, dev = q.dtype, cache.device
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q must be float16 or bfloat16")
    if cache.dtype != "e2m1" and cache.dtype != dtype:
        raise TypeError(f"q must be {cache.dtype} as the cache, got {dtype}")
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    _need_bend(scale, softcap)
    if max_rows is not None and max_rows < 1:
        raise ValueError(f"max_rows must be positive, got {max_rows}")
    if prefix_lens is not None and not causal:
        raise ValueError("prefix_lens belongs to causal attention")
    shape = q.shape
    tokens, heads, dim = shape
    if dim != cache.head_dim or heads < 1 or heads % cache.kv_heads:
        raise ValueError(f"q's {heads} heads of {dim} cannot share the cache's {cache.kv_heads} of {cache.head_dim}")
    q_token, q_head = _head_rows(q, "q", shape, dtype, dev)
    pool, batch = _pool(cache, block_table, kv_lens)
    offsets = _offsets(q_offsets, batch, tokens, dev)
    if out is None:
        out = torch.empty_like(q)
        out_token, out_head, _ = out.stride()
    else:
        out_token, out_head = _head_rows(out, "out", shape, dtype, dev)
    if lse is None:
        lse = torch.empty((heads, tokens), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", device=dev, dtypes=(torch.float32,), numel=heads * tokens)
    slope_ptr = 0
    if slopes is not None:
        _need(slopes, "slopes", device=dev, dtypes=(torch.float32,), numel=heads)
        slope_ptr = slopes.data_ptr()
    prefix = _list(prefix_lens, "prefix_lens", batch, dev)

    # The size depends on sizes and on which lists there are, not on any value.
    key = (cache.dtype, cache.kv_heads, cache.page_size, shape, batch, block_table.shape[1], max_rows, offsets == 0)
    need = block._sizes.get(("h3qk_cache_attention_workspace_bytes", dev.index, key))
    call = [_DTYPES[dtype], heads, 1 if causal else 0, min(max_rows or 0, 1 << 30), scale or 0.0, softcap, tokens,
            q.data_ptr(), out.data_ptr(), q_token, q_head, out_token, out_head, lse.data_ptr(), slope_ptr, prefix, offsets]
    if need is None:
        need = block._size("h3qk_cache_attention_workspace_bytes", dev, pool, _ATTN.pack(*call, 0, 0), key=key)
    ws = ws_bytes = 0
    if need:
        workspace, ws_bytes = _workspace(workspace, need, dev)
        ws = workspace.data_ptr()
    block._call("h3qk_cache_attention", dev, pool, _ATTN.pack(*call, ws, ws_bytes), _stream(dev))
    return out, lse


@_on_stream
def cache_read(cache, block_table, kv_lens, *, starts=None, rows: int | None = None, dtype=None, out_k=None, out_v=None):
    """Rows of a cache as dense tensors (h3qk_cache_read): (k, v), each
    [batch, kv_heads, rows, head_dim], with rows ``starts`` (int32 [batch],
    default 0) to ``kv_lens`` of each sequence, at most ``rows`` of them
    (default: all that the table has room for), and zeros after them.
    ``dtype`` is a 16-bit cache's own; 4-bit values come in float16 or bfloat16
    (default).  ``attention`` takes them as its k, v."""
    pool, batch = _pool(cache, block_table, kv_lens)
    dev = cache.device
    if dtype is None:
        dtype = torch.bfloat16 if cache.dtype == "e2m1" else cache.dtype
    if dtype not in (torch.float16, torch.bfloat16) or cache.dtype not in ("e2m1", dtype):
        raise TypeError(f"a {cache.dtype} cache cannot be read as {dtype}")
    if rows is None:
        rows = block_table.shape[1] * cache.page_size
    if rows < 0 or rows >= 1 << 30:
        raise ValueError(f"rows must be from 0 to 2^30, got {rows}")
    first = _list(starts, "starts", batch, dev)
    shape = (batch, cache.kv_heads, rows, cache.head_dim)
    if out_k is None:
        out_k = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _need(out_k, "out_k", device=dev, dtypes=(dtype,), numel=batch * cache.kv_heads * rows * cache.head_dim)
    if out_v is None:
        out_v = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _need(out_v, "out_v", device=dev, dtypes=(dtype,), numel=batch * cache.kv_heads * rows * cache.head_dim)
    block._call("h3qk_cache_read", dev, pool, first, rows, _DTYPES[dtype], out_k.data_ptr(), out_v.data_ptr(), _stream(dev))
    return out_k, out_v
