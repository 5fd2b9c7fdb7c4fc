"""Python binding of the attention block's operators: layer norm and its
gradient, the gradient of the fused QK preparation, and attention.

As in ``h3qk``, this only checks tensors and passes their addresses: each
operator runs in the library's CUDA kernels on the current stream, or on the
one passed as ``stream`` (the call then behaves as if it were the current
one), and workspaces come from torch's allocator unless the caller passes one.

The results carry no autograd graph: in training the forward and its
``..._backward`` are the two halves of a torch.autograd.Function
(examples/attention_block.py has one for each operator).  Incoming gradients
may be expanded tensors, as autograd makes them; such are copied first.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import h3qk
from .h3qk import BF16, FP16, OK, H3QKError, _need, _need_common, _opts_for, _ptr

FP32 = 4
_DTYPES = {torch.float16: FP16, torch.bfloat16: BF16, torch.float32: FP32}
_P, _I32, _I64, _SZ, _F, _INT = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float,
                                 ctypes.c_int)

_SIGNATURES = {
    "h3qk_layer_norm": (_INT, [_P, _INT, _I64, _I32, _I64, _P, _P, _I64, _F, _P, _P, _P]),
    "h3qk_layer_norm_backward_workspace_bytes": (_SZ, [_I64, _I32, _I64]),
    "h3qk_layer_norm_backward": (_INT, [_P, _I64, _P, _INT, _I64, _I32, _I64, _P, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "h3qk_attention_workspace_bytes": (_SZ, [ctypes.c_char_p]),
    "h3qk_attention": (_INT, [ctypes.c_char_p, _P]),
    "h3qk_attention_backward_workspace_bytes": (_SZ, [ctypes.c_char_p]),
    "h3qk_attention_backward": (_INT, [ctypes.c_char_p, _P]),
    "h3qk_attention_stuck": (_I64, []),
    "h3qk_prepare_backward_workspace_bytes": (_SZ, [_I32]),
    "h3qk_prepare_backward": (_INT, [_P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I64, _P, _P, _P, _P, _SZ,
                                     ctypes.POINTER(h3qk.Opts), _P]),
}


_functions = {}   # name -> (library, function): a reloaded library gets its own
_sizes = {}       # workspace sizes by entry point, device and shape


def _fn(name):
    L = h3qk.lib()
    known = _functions.get(name)
    if known is None or known[0] is not L:
        f = getattr(L, name)
        f.restype, f.argtypes = _SIGNATURES[name]
        known = _functions[name] = (L, f)
    return known[1]


# The current stream's address without the Stream object around it (2 us less
# a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _on_stream(f):
    """Runs an operator with ``stream`` (a torch stream or a raw address) as
    torch's current one, so that what it allocates, its workspace above all,
    belongs to that stream and is not given away while the kernels still run."""

    @functools.wraps(f)
    def run(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return f(*args, **kw)

    return run


def _call(name, dev, *args):
    """A library call with the tensors' device current (the library keys its
    caches on it)."""
    f = _fn(name)
    if dev.type != "cuda":
        raise ValueError(f"{name} takes CUDA tensors, got {dev}")
    if dev.index == torch.cuda.current_device():
        st = f(*args)
    else:
        with torch.cuda.device(dev):
            st = f(*args)
    if st != OK:
        raise H3QKError(st, h3qk.status_string(st), int(h3qk.lib().h3qk_last_cuda_error()), name)


def _size(name, dev, *args, key=None):
    """A workspace size, asked once per device and shape (the arguments, or
    ``key``) with the tensors' device current."""
    at = (name, dev.index, key or args)
    n = _sizes.get(at)
    if n is None:
        if dev.index == torch.cuda.current_device():
            n = _fn(name)(*args)
        else:
            with torch.cuda.device(dev):
                n = _fn(name)(*args)
        if len(_sizes) > 4096:
            _sizes.clear()
        _sizes[at] = n
    return n


def _workspace(workspace, nbytes, dev):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev), nbytes
    _need(workspace, "workspace", device=dev)
    return workspace, workspace.numel() * workspace.element_size()


def _spread(grad):
    """A gradient that autograd hands over expanded (one value for many
    elements, as the sum of an output gives), written out; others as they are."""
    return grad.contiguous() if grad is not None and 0 in grad.stride() else grad


def _need_rows(x, name, dtypes):
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {x.dtype}")
    if x.dim() == 2 and x.is_contiguous():
        return
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D [rows, width] with unit inner stride")
    if x.shape[0] > 1 and x.stride(0) < x.shape[1]:
        raise ValueError(f"{name} must not have overlapping rows")


def _row_stride(x):
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _need_affine(w, name, width, batch, dev):
    """The groups a weight stands for: [width] is shared, [batch, width] has a row per item."""
    if w.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {w.dtype}")
    if w.shape != (width,) and w.shape != (batch, width):
        raise ValueError(f"{name} must have shape ({width},) or ({batch}, {width}), got {tuple(w.shape)}")
    if not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if w.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {w.device}")
    return 1 if w.dim() == 1 else batch


@_on_stream
def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-6, batch: int = 1, out=None, stats=None):
    """Layer norm of the rows of x [rows, width] (float16, bfloat16 or
    float32; any row stride >= width).  ``weight`` and ``bias`` are float32
    [width], or [batch, width] with one row per item of rows / batch rows (an
    adaptive norm).  Returns (y, stats): y [rows, width] of x's type, stats
    float32 [rows, 2] with each row's mean and reciprocal deviation, which
    ``layer_norm_backward`` reads (h3qk_layer_norm)."""
    _need_rows(x, "x", _DTYPES)
    rows, width = x.shape
    dev = x.device
    if batch < 1 or rows % batch:
        raise ValueError("rows must be a multiple of batch")
    groups = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            g = _need_affine(t, name, width, batch, dev)
            if groups is not None and g != groups:
                raise ValueError("weight and bias must have the same shape")
            groups = g
    if out is None:
        out = torch.empty((rows, width), dtype=x.dtype, device=dev)
    else:
        _need(out, "out", device=dev, dtypes=(x.dtype,), numel=rows * width)
    if stats is None:
        stats = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    else:
        _need(stats, "stats", device=dev, dtypes=(torch.float32,), numel=2 * rows)
    _call("h3qk_layer_norm", dev, x.data_ptr(), _DTYPES[x.dtype], rows, width, _row_stride(x), _ptr(weight), _ptr(bias),
          groups or 1, eps, out.data_ptr(), stats.data_ptr(), _stream(dev))
    return out, stats


@_on_stream
def layer_norm_backward(grad_out, x, weight, stats, *, batch: int = 1, need_weight_grad: bool = True, out=None,
                        grad_weight=None, grad_bias=None, workspace=None):
    """The gradient of ``layer_norm``: grad_out [rows, width] of x's type, x
    and weight as the forward took them, stats as it returned them.  Returns
    (grad_x, grad_weight, grad_bias); the last two are float32 of the
    weight's shape, summed over the rows that share them, or None without a
    weight or with ``need_weight_grad=False`` (h3qk_layer_norm_backward)."""
    grad_out = _spread(grad_out)
    _need_rows(x, "x", _DTYPES)
    _need_rows(grad_out, "grad_out", (x.dtype,))
    rows, width = x.shape
    dev = x.device
    if tuple(grad_out.shape) != (rows, width) or grad_out.device != dev:
        raise ValueError(f"grad_out must have shape ({rows}, {width}) on {dev}")
    if batch < 1 or rows % batch:
        raise ValueError("rows must be a multiple of batch")
    _need(stats, "stats", device=dev, dtypes=(torch.float32,), numel=2 * rows)
    groups = 1 if weight is None else _need_affine(weight, "weight", width, batch, dev)
    if out is None:
        out = torch.empty((rows, width), dtype=x.dtype, device=dev)
    else:
        _need(out, "out", device=dev, dtypes=(x.dtype,), numel=rows * width)
    sums = weight is not None and need_weight_grad
    ws_bytes = 0
    if sums:
        if grad_weight is None:
            grad_weight = torch.empty_like(weight)
        if grad_bias is None:
            grad_bias = torch.empty_like(weight)
        for t, name in ((grad_weight, "grad_weight"), (grad_bias, "grad_bias")):
            _need(t, name, device=dev, dtypes=(torch.float32,), numel=groups * width)
        workspace, ws_bytes = _workspace(
            workspace, _size("h3qk_layer_norm_backward_workspace_bytes", dev, rows, width, groups), dev)
    else:
        grad_weight = grad_bias = workspace = None
    _call("h3qk_layer_norm_backward", dev, grad_out.data_ptr(), _row_stride(grad_out), x.data_ptr(), _DTYPES[x.dtype],
          rows, width, _row_stride(x), _ptr(weight), groups, stats.data_ptr(), out.data_ptr(), _ptr(grad_weight),
          _ptr(grad_bias), _ptr(workspace), ws_bytes, _stream(dev))
    return out, grad_weight, grad_bias


@_on_stream
def prepare_backward(grad_q, grad_k, grad_v, qkv, norm_wq, norm_wk, positions, *, heads: int, head_dim: int,
                     rotary_dim: int, batch: int = 1, valid_len: int | None = None, n_axes: int | None = None,
                     axis_dims=None, theta: float = 10000.0, eps: float = 1e-6, out=None, grad_wq=None, grad_wk=None,
                     workspace=None, layout: str = "head_major", valid_lens=None):
    """The gradient of a 16-bit ``prepare`` call.  grad_q, grad_k, grad_v are
    contiguous [batch, heads, S, head_dim] (or [batch, S, heads, head_dim]
    with ``layout="token_major"``) of qkv's type; the other arguments are the
    forward call's.  Returns (grad_qkv, grad_wq, grad_wk): grad_qkv
    [tokens, 3*heads*head_dim] of qkv's type, zero in rows past the valid
    prefix, and the float32 [head_dim] weight gradients
    (h3qk_prepare_backward)."""
    if qkv.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("qkv must be float16 or bfloat16")
    if qkv.dim() != 2 or qkv.stride(1) != 1:
        raise ValueError("qkv must be 2-D [tokens, row_stride] with unit inner stride")
    tokens = qkv.shape[0]
    if tokens % batch:
        raise ValueError("tokens must be a multiple of batch")
    seq = tokens // batch
    if valid_len is None:
        valid_len = seq
    if n_axes is None:
        n_axes = positions.shape[1] if positions is not None and positions.dim() == 2 else 3
    dev = qkv.device
    _need_common(qkv, norm_wq, norm_wk, positions, tokens=tokens, heads=heads, head_dim=head_dim,
                 rotary_dim=rotary_dim, n_axes=n_axes, batch=batch, valid_lens=valid_lens, device=dev)
    n = tokens * heads * head_dim
    grad_q, grad_k, grad_v = _spread(grad_q), _spread(grad_k), _spread(grad_v)
    for t, name in ((grad_q, "grad_q"), (grad_k, "grad_k"), (grad_v, "grad_v")):
        _need(t, name, device=dev, dtypes=(qkv.dtype,), numel=n)
    if out is None:
        out = torch.empty((tokens, 3 * heads * head_dim), dtype=qkv.dtype, device=dev)
    else:
        _need(out, "out", device=dev, dtypes=(qkv.dtype,), numel=3 * n)
    if grad_wq is None:
        grad_wq = torch.empty(head_dim, dtype=torch.float32, device=dev)
    if grad_wk is None:
        grad_wk = torch.empty(head_dim, dtype=torch.float32, device=dev)
    for t, name in ((grad_wq, "grad_wq"), (grad_wk, "grad_wk")):
        _need(t, name, device=dev, dtypes=(torch.float32,), numel=head_dim)
    o = _opts_for(qkv, n_axes=n_axes, axis_dims=axis_dims, theta=theta, eps=eps, batch=batch)
    o.out_layout = {"head_major": h3qk.HEAD_MAJOR, "token_major": h3qk.TOKEN_MAJOR}[layout]
    o.valid_lens = _ptr(valid_lens)
    workspace, ws_bytes = _workspace(workspace, _size("h3qk_prepare_backward_workspace_bytes", dev, head_dim), dev)
    _call("h3qk_prepare_backward", dev, grad_q.data_ptr(), grad_k.data_ptr(), grad_v.data_ptr(), qkv.data_ptr(),
          norm_wq.data_ptr(), norm_wk.data_ptr(), _ptr(positions), tokens, heads, head_dim, rotary_dim, valid_len,
          out.data_ptr(), grad_wq.data_ptr(), grad_wk.data_ptr(), workspace.data_ptr(), ws_bytes, ctypes.byref(o),
          _stream(dev))
    return out, grad_wq, grad_wk


# h3qk_attn (include/h3qk.h), packed in one step
_ATTN = struct.Struct("@8i2f2q16PN24q")
_NO_STRIDES = (0, 0, 0)


def _need_heads(t, name, shape, dtype, dev):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    st = t.stride()
    if st[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return st[:3]


def _need_lens(t, name, n, dev):
    if t is None:
        return 0
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}, got shape {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return t.data_ptr()


# What binary32 does not round to zero or infinity lies between these.
_F32_LOW, _F32_HIGH = 2.0 ** -150, 2.0 ** 128 - 2.0 ** 103


def _need_bend(scale, softcap):
    """Refuses what the library would refuse, or what binary32 makes a zero, which it reads as a default.  The size
    of a workspace is kept for calls that differ in these only, so none is asked with a value that is refused."""
    if scale is not None and not _F32_LOW < scale < _F32_HIGH:
        raise ValueError(f"scale must be positive and finite (in binary32), got {scale}")
    if softcap != 0.0 and not _F32_LOW < softcap < _F32_HIGH:
        raise ValueError(f"softcap must be 0, or positive and finite (in binary32), got {softcap}")


def _attn_common(q, k, v, scale, softcap, slopes, prefix_lens, doc_offsets, q_lens, kv_lens, q_starts):
    """Checks shared by both directions: (batch, heads, kv_heads, q_rows, kv_rows, dim, docs, strides, pointers)."""
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q must be float16 or bfloat16")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be [batch, heads, rows, head_dim]")
    _need_bend(scale, softcap)
    dev = q.device
    batch, heads, sq, dim = q.shape
    _, kv_heads, sk, _ = k.shape
    if kv_heads == 0 or heads % kv_heads:
        raise ValueError(f"{heads} heads cannot share {kv_heads} K/V heads")
    strides = (_need_heads(q, "q", (batch, heads, sq, dim), q.dtype, dev),
               _need_heads(k, "k", (batch, kv_heads, sk, dim), q.dtype, dev),
               _need_heads(v, "v", (batch, kv_heads, sk, dim), q.dtype, dev))
    docs = 0
    if doc_offsets is not None:
        docs = doc_offsets.shape[0] - 1 if doc_offsets.dim() == 1 else 0
        if docs < 1:
            raise ValueError("doc_offsets must be a vector of at least two offsets")
        if batch != 1 or sq != sk:
            raise ValueError("documents are packed along the rows of one item, the same for queries and keys")
        if q_lens is not None or kv_lens is not None or q_starts is not None:
            raise ValueError("doc_offsets excludes q_lens, kv_lens and q_starts")
    slope_ptr = 0
    if slopes is not None:
        _need(slopes, "slopes", device=dev, dtypes=(torch.float32,), numel=heads)
        slope_ptr = slopes.data_ptr()
    lists = (slope_ptr, _need_lens(prefix_lens, "prefix_lens", docs or batch, dev),
             _need_lens(doc_offsets, "doc_offsets", docs + 1, dev), _need_lens(q_lens, "q_lens", batch, dev),
             _need_lens(kv_lens, "kv_lens", batch, dev), _need_lens(q_starts, "q_starts", batch, dev))
    return batch, heads, kv_heads, sq, sk, dim, docs, strides, lists


@_on_stream
def attention(q, k, v, *, scale: float | None = None, softcap: float = 0.0, slopes=None, causal: bool = False,
              prefix_lens=None, doc_offsets=None, q_lens=None, kv_lens=None, q_starts=None, out=None, lse=None,
              workspace=None):
    """Attention on head rows as ``prepare`` writes them.

    q: float16/bfloat16 [batch, heads, Sq, D]; k, v: [batch, kv_heads, Sk, D]
    of the same type, kv_heads dividing heads (head h reads K/V head
    h // (heads // kv_heads)), D a multiple of 8 up to 128.  Any batch, head
    and row strides that are multiples of 8 elements will do, so a token-major
    tensor is passed as its ``transpose(1, 2)`` and a cache as a slice.

    Scores are scale * q.k (default 1 / sqrt(D)), bent to softcap * tanh(z /
    softcap) when ``softcap`` is positive, less ``slopes[h]`` (float32
    [heads]) times the distance of query and key.  A row sees the keys below
    its item's ``kv_lens`` (int32 [batch]); with ``causal`` of those only the
    ones up to its own position, and the first ``prefix_lens`` of them (int32
    [batch], or one per document).  ``q_lens`` limits the rows that attend;
    ``q_starts`` is row 0's position among the keys (default: 0 when Sq == Sk,
    else kv_len - q_len).  ``doc_offsets`` (int32 [n + 1], from 0) packs n
    documents along the rows of one item: each attends within itself.

    Returns (out, lse): out like q, lse float32 [batch, heads, Sq], the
    natural logarithm of each row's sum of exponentials.  Rows that see
    nothing have out = 0 and lse = -inf.  A call with few rows per K/V head
    (tokens produced one by one) splits the keys over the GPU and joins the
    parts (h3qk_attention)."""
    batch, heads, kv_heads, sq, sk, dim, docs, strides, lists = _attn_common(
        q, k, v, scale, softcap, slopes, prefix_lens, doc_offsets, q_lens, kv_lens, q_starts)
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    out_strides = _need_heads(out, "out", (batch, heads, sq, dim), q.dtype, dev)
    if lse is None:
        lse = torch.empty((batch, heads, sq), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", device=dev, dtypes=(torch.float32,), numel=batch * heads * sq)

    def args(ws, ws_bytes):
        return _ATTN.pack(_DTYPES[q.dtype], batch, heads, kv_heads, dim, 1 if causal else 0, docs, 0, scale or 0.0,
                          softcap, sq, sk, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                          0, 0, 0, 0, *lists, ws, ws_bytes, *strides[0], *strides[1], *strides[2], *out_strides,
                          *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES)

    # The size depends on the sizes, the masks' kind and which lists there are
    # (the library does not read them), not on any value.
    shape = (batch, heads, kv_heads, sq, sk, dim, bool(causal), docs, *(t != 0 for t in lists))
    need = _sizes.get(("h3qk_attention_workspace_bytes", dev.index, shape))
    if need is None:
        need = _size("h3qk_attention_workspace_bytes", dev, args(0, 0), key=shape)
    ws = ws_bytes = 0
    if need:
        workspace, ws_bytes = _workspace(workspace, need, dev)
        ws = workspace.data_ptr()
    _call("h3qk_attention", dev, args(ws, ws_bytes), _stream(dev))
    return out, lse


@_on_stream
def attention_backward(grad_out, q, k, v, out, lse, *, scale: float | None = None, softcap: float = 0.0, slopes=None,
                       causal: bool = False, prefix_lens=None, doc_offsets=None, q_lens=None, kv_lens=None,
                       q_starts=None, grad_q=None, grad_k=None, grad_v=None, workspace=None):
    """The gradient of ``attention``: grad_out like out, the forward's q, k, v
    and keyword arguments, out and lse as it returned them.  Returns (grad_q,
    grad_k, grad_v) like q, k and v; heads that share a K/V head add to one
    gradient, and rows and keys that take no part get zeros.  The same call
    gives the same bits every time.  The slopes get no gradient
    (h3qk_attention_backward)."""
    batch, heads, kv_heads, sq, sk, dim, docs, strides, lists = _attn_common(
        q, k, v, scale, softcap, slopes, prefix_lens, doc_offsets, q_lens, kv_lens, q_starts)
    grad_out = _spread(grad_out)
    dev = q.device
    row, key = (batch, heads, sq, dim), (batch, kv_heads, sk, dim)
    out_strides = _need_heads(out, "out", row, q.dtype, dev)
    do_strides = _need_heads(grad_out, "grad_out", row, q.dtype, dev)
    _need(lse, "lse", device=dev, dtypes=(torch.float32,), numel=batch * heads * sq)
    grad_q = torch.empty_like(q) if grad_q is None else grad_q
    grad_k = torch.empty_like(k) if grad_k is None else grad_k
    grad_v = torch.empty_like(v) if grad_v is None else grad_v
    dq_strides = _need_heads(grad_q, "grad_q", row, q.dtype, dev)
    dk_strides = _need_heads(grad_k, "grad_k", key, q.dtype, dev)
    dv_strides = _need_heads(grad_v, "grad_v", key, q.dtype, dev)
    # one binary32 word a row, as h3qk_attention_backward_workspace_bytes says
    workspace, ws_bytes = _workspace(workspace, (batch * heads * sq * 4 + 15) // 16 * 16, dev)
    packed = _ATTN.pack(_DTYPES[q.dtype], batch, heads, kv_heads, dim, 1 if causal else 0, docs, 0, scale or 0.0, softcap,
                        sq, sk, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                        grad_out.data_ptr(), grad_q.data_ptr(), grad_k.data_ptr(), grad_v.data_ptr(), *lists,
                        workspace.data_ptr(), ws_bytes, *strides[0], *strides[1], *strides[2], *out_strides, *do_strides,
                        *dq_strides, *dk_strides, *dv_strides)
    _call("h3qk_attention_backward", dev, packed, _stream(dev))
    return grad_q, grad_k, grad_v
