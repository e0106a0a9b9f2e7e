"""Python binding of the operators of libgnsilu (``include/gnsilu.h``) that serve
from a paged cache in 8 bits: RMS norm with the residual's addition and an output
in 8 bits (and its backward pass), appending new tokens to the cache with the
rotary positions applied on the way, and attention over the cache.

The conventions are those of ``block``: every step runs in the library's kernels,
unsupported input gives ``None``, a CUDA or kernel failure raises ``GnError``, and
``stream`` is a ``torch.cuda.Stream`` to run on instead of the current one.

Calls can be captured into CUDA graphs.  The first call of a process on a device sets the
library up there (a status word in mapped memory) and has to come ahead of a capture.

The cache belongs to the caller, as plain tensors:

* ``k_pages`` and ``v_pages``, ``torch.float8_e4m3fn`` [pages, page_size, Hk, D], any
  order of the first three axes in memory (a head's tokens of a page next to each
  other read fastest: ``torch.zeros(pages, Hk, page_size, D, ...).transpose(1, 2)``);
* ``k_scales`` and ``v_scales``, fp32 [pages, Hk]: an element is its byte's value times
  its page's and head's scale, which is not negative;
* ``table``, int32 [sequences, width]: the pages of every sequence in order;
* ``lengths``, int32 [sequences]: the tokens of every sequence, the new ones of the call
  among them.
"""
from __future__ import annotations

import ctypes
import math
import struct

from .block import (MAX_AXES, _Torch, _axes_array, _ends_like, _head_strides, _heads_like, _like, _packed_strides,
                    _param_format, _ptr, _row_strides, _run, _start, _wants_grad)
from .gnsilu import _finish


class _Eight:
    """The 8-bit type, from the first call on."""
    kind = None

    @classmethod
    def get(cls, T):
        if cls.kind is None:
            cls.kind = T.torch.float8_e4m3fn
        return cls.kind


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
_Strides8 = struct.Struct("8q")


def gn_rms_norm_workspace_bytes(rows: int, cols: int) -> int:
    return int(_start()[0].gn_rms_norm_workspace_bytes(rows, cols))


def _rows_of(shape, tensors):
    """(inner, the strides of each tensor or (0, 0) without one, ...), or None."""
    there = [t for t in tensors if t is not None]
    rows_at = _row_strides(shape, there)
    if rows_at is None:
        return None
    inner, found = rows_at
    found, strides = iter(found), []
    for t in tensors:
        strides += (0, 0) if t is None else (next(found), next(found))
    return inner, strides


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, quantize: bool = False, out=None, total_out=None,
             stream=None):
    """RMS norm over the last axis of a bf16, fp16 or fp32 CUDA tensor [..., C], C up to
    16384, of ``total`` = x + residual: ``(y, scales, total, rstd)``, or None when not
    supported.

    ``residual`` (like x): the residual stream; total, rounded to x's dtype, is what the
    stream goes on with (``total_out`` if given; it may be residual or x).  Without one
    total is x itself.  ``weight``: a contiguous [C] tensor of any of the three dtypes.
    y is shaped like x (``out`` if given; without a residual it may be x).  ``quantize``: y
    is float8_e4m3fn of the normed rows over fp32 ``scales`` shaped ``x.shape[:-1]``, a
    row's largest magnitude over 448; scales is None otherwise.  rstd (fp32) is for
    ``rms_norm_backward``.  Strides as for ``layer_norm``."""
    L, T = _start()
    if not (isinstance(x, T.Tensor) and x.is_cuda):
        return None
    shape, device, kind = x.shape, x.device, T.formats.get(x.dtype)
    if kind is None or not shape or shape[-1] < 1 or _wants_grad(x, weight, residual):
        return None
    cols, wkind = shape[-1], 0
    if weight is not None:
        wkind = _param_format(weight, cols, device, T)
        if wkind is None:
            return None
    if residual is None:
        if total_out is not None:
            return None
    elif not _like(residual, x, T) or (total_out is not None and not _like(total_out, x, T)):
        return None
    y_kind = _Eight.get(T) if quantize else x.dtype
    if out is not None and not (isinstance(out, T.Tensor) and out.shape == shape and out.dtype == y_kind and out.device == device):
        return None
    if out is None and total_out is None and x.is_contiguous() and (residual is None or residual.is_contiguous()):
        inner, strides = 0, (0, cols) * 4
    else:
        packed = _packed_strides(shape)
        rows_at = _rows_of(shape, (x.stride(), None if residual is None else residual.stride(),
                                   packed if out is None else out.stride(),
                                   None if residual is None else packed if total_out is None else total_out.stride()))
        if rows_at is None:
            return None
        inner, strides = rows_at

    def go(handle):
        y = T.empty(shape, dtype=y_kind, device=device) if out is None else out
        total = None
        if residual is not None:
            total = T.empty(shape, dtype=x.dtype, device=device) if total_out is None else total_out
        rstd = T.empty(shape[:-1], dtype=T.float32, device=device)
        scales = T.empty(shape[:-1], dtype=T.float32, device=device) if quantize else None
        rc = L.gn_rms_norm(x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(), _ptr(total), _ptr(scales),
                           rstd.data_ptr(), rstd.numel(), cols, inner or max(1, rstd.numel()), _Strides8.pack(*strides), eps,
                           kind, wkind, handle)
        return (y, scales, x if total is None else total, rstd) if rc == 0 or _finish(rc, "gn_rms_norm") else None
    return _run(device, stream, (x, weight, residual, out, total_out), go)


def rms_norm_backward(dy, total, rstd, weight=None, dtotal=None, out=None, stream=None):
    """Backward pass of ``rms_norm`` (with y in x's dtype): ``(dx, dweight)`` from the gradient
    dy of y, what the norm was taken of (``total``, x without a residual) and rstd as it
    returned them, its weight, and the gradient ``dtotal`` that the residual stream sends
    back (or None).  dx is the gradient of x and of the residual alike (``out`` if given;
    it may be dy, total or dtotal); dweight has the weight's dtype and is None without
    one.  None when not supported."""
    L, T = _start()
    if not (isinstance(total, T.Tensor) and total.is_cuda):
        return None
    shape, device, kind = total.shape, total.device, T.formats.get(total.dtype)
    if kind is None or not shape or shape[-1] < 1 or not _like(dy, total, T) or _wants_grad(dy, total, weight, dtotal):
        return None
    if not (isinstance(rstd, T.Tensor) and rstd.dtype == T.float32 and rstd.shape == shape[:-1] and rstd.is_contiguous()
            and rstd.device == device):
        return None
    cols, wkind = shape[-1], 0
    if weight is not None:
        wkind = _param_format(weight, cols, device, T)
        if wkind is None:
            return None
    if (dtotal is not None and not _like(dtotal, total, T)) or (out is not None and not _like(out, total, T)):
        return None
    if out is None and total.is_contiguous() and dy.is_contiguous() and (dtotal is None or dtotal.is_contiguous()):
        inner, strides = 0, (0, cols) * 4
    else:
        rows_at = _rows_of(shape, (dy.stride(), total.stride(), None if dtotal is None else dtotal.stride(),
                                   _packed_strides(shape) if out is None else out.stride()))
        if rows_at is None:
            return None
        inner, strides = rows_at

    def go(handle):
        dx = T.empty(shape, dtype=total.dtype, device=device) if out is None else out
        rows = rstd.numel()
        dw = workspace = None
        need = 0
        if weight is not None:
            dw = T.torch.empty_like(weight)
            need = max(1, L.gn_rms_norm_workspace_bytes(rows, cols))
            workspace = T.empty(need, dtype=T.uint8, device=device)
        rc = L.gn_rms_norm_backward(dy.data_ptr(), total.data_ptr(), _ptr(weight), rstd.data_ptr(), _ptr(dtotal),
                                    dx.data_ptr(), _ptr(dw), rows, cols, inner or max(1, rows), _Strides8.pack(*strides), kind,
                                    wkind, _ptr(workspace), need, handle)
        return (dx, dw) if rc == 0 or _finish(rc, "gn_rms_norm_backward") else None
    return _run(device, stream, (dy, total, rstd, weight, dtotal, out), go)


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------
# gn_cache, gn_append_args and gn_attn_cached_args of include/gnsilu.h
_CACHE = struct.Struct("4P6q3P2q4i")
_APPEND = struct.Struct("4P9q2Pd5i4x")
_ATTN = struct.Struct("4P3q2f3i4x")


def _pool_strides(shape, strides):
    """Page, token and head stride; of an axis of length one the packed ones."""
    pages, size, heads, dim = shape
    page, token, head, _ = strides
    if heads == 1:
        head = dim
    if size == 1:
        token = heads * dim
    if pages == 1:
        page = size * heads * dim
    return page, token, head


def _cache_args(k_pages, v_pages, k_scales, v_scales, table, lengths, cu, T):
    """(The packed gn_cache, the pools' shape, device), or None if not supported."""
    if not (isinstance(k_pages, T.Tensor) and k_pages.is_cuda and k_pages.dtype == _Eight.get(T)):
        return None
    shape, device = k_pages.shape, k_pages.device
    if len(shape) != 4 or not _like(v_pages, k_pages, T) or 0 in shape:
        return None
    ks, vs = k_pages.stride(), v_pages.stride()
    if shape[3] > 1 and (ks[3] != 1 or vs[3] != 1):
        return None
    for t in (k_scales, v_scales):
        if not (isinstance(t, T.Tensor) and t.dtype == T.float32 and t.device == device and t.shape == (shape[0], shape[2])
                and t.is_contiguous()):
            return None
    if not (isinstance(table, T.Tensor) and table.dtype == T.int32 and table.device == device and table.dim() == 2
            and table.is_contiguous()):
        return None
    sequences, width = table.shape
    if sequences < 1 or width < 1 or not _ends_like(lengths, sequences, device, T):
        return None
    if cu is not None and not _ends_like(cu, sequences + 1, device, T):
        return None
    if sequences > 1 << 20 or shape[0] >= 1 << 31 or max(shape[1], shape[2], shape[3]) >= 1 << 20:
        return None
    return _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                       *_pool_strides(shape, ks), *_pool_strides(shape, vs), table.data_ptr(), lengths.data_ptr(),
                       0 if cu is None else cu.data_ptr(), shape[0], width, sequences, shape[1], shape[2],
                       shape[3]), shape, device


def cache_append(k, v, k_pages, v_pages, k_scales, v_scales, table, lengths, cu=None, q=None, positions=None, axes_dim=(),
                 theta: float = 10000.0, interleaved: bool = True, out=None, stream=None):
    """Appends the new tokens' keys k and values v [T, Hk, D] (bf16, fp16 or fp32, channels
    contiguous) to the cache (see the module), in place: True, or the turned query heads
    with ``q``; None when not supported.

    Sequence s owns the packed tokens [cu[s], cu[s + 1]) (``cu``: int32 [sequences + 1] on
    the GPU; None: T / sequences each), the last of which is its token lengths[s] - 1.
    ``positions`` [T, axes], ``axes_dim``, ``theta`` and ``interleaved`` turn the keys, and
    the query heads q [T, H, D], as ``rope_nd`` does (None: nothing turns); sum(axes_dim) is
    at most D.  ``out``: where the turned query heads go (it may be q).

    page_size is a multiple of 8 up to 256, D of 16 up to 128.  A page's scale is the least
    power of two with which its largest magnitude is at most 448; where a new token needs a larger
    one, the page's other tokens are rounded to it.  A page that the call appends to
    belongs to one sequence.  Tokens of no sequence, or past the table, are not stored."""
    L, T = _start()
    found = _cache_args(k_pages, v_pages, k_scales, v_scales, table, lengths, cu, T)
    if found is None or not isinstance(k, T.Tensor):
        return None
    cache, pool, device = found
    dtype = k.dtype
    kind = T.formats.get(dtype)
    if kind is None or _wants_grad(q, k, v) or not _heads_like(k, dtype, device, T) or not _heads_like(v, dtype, device, T):
        return None
    shape = k.shape
    if v.shape != shape or shape[1:] != pool[2:]:
        return None
    place, axes_dim = 0, tuple(axes_dim)
    if positions is not None:
        if not (isinstance(positions, T.Tensor) and positions.device == device and positions.is_contiguous()
                and positions.shape == (shape[0], len(axes_dim)) and 1 <= len(axes_dim) <= MAX_AXES):
            return None
        place = T.positions.get(positions.dtype)
        if place is None:
            return None
    elif axes_dim:
        return None
    q_strides, heads = (0, 0), 0
    if q is not None:
        if not _heads_like(q, dtype, device, T) or q.shape[0] != shape[0] or q.shape[2] != shape[2] or q.shape[1] > 1 << 16:
            return None
        q_strides, heads = _head_strides(q.shape, q.stride()), q.shape[1]
        if out is not None and not (_heads_like(out, dtype, device, T) and out.shape == q.shape):
            return None
    elif out is not None:
        return None

    def go(handle):
        to, to_strides = out, (0, 0)
        if q is not None:
            if out is None:
                to, to_strides = T.empty(q.shape, dtype=dtype, device=device), (heads * shape[2], shape[2])
            else:
                to_strides = _head_strides(q.shape, out.stride())
        axes = _axes_array(axes_dim) if axes_dim else None
        args = _APPEND.pack(0 if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), 0 if to is None else to.data_ptr(),
                            *q_strides, *_head_strides(shape, k.stride()), *_head_strides(shape, v.stride()), *to_strides,
                            shape[0], 0 if positions is None else positions.data_ptr(),
                            0 if axes is None else ctypes.addressof(axes), theta, heads, len(axes_dim), place, bool(interleaved),
                            kind)
        rc = L.gn_cache_append(cache, args, handle)
        return (True if to is None else to) if rc == 0 or _finish(rc, "gn_cache_append") else None
    return _run(device, stream, (k, v, k_pages, v_pages, k_scales, v_scales, table, lengths, cu, q, positions, out), go)


def gn_attn_cached_workspace_bytes(tokens: int, sequences: int, heads: int, kv_heads: int, dim: int) -> int:
    return int(_start()[0].gn_attn_cached_workspace_bytes(tokens, sequences, heads, kv_heads, dim))


def attention_cached(q, k_pages, v_pages, k_scales, v_scales, table, lengths, cu=None, causal: bool = True, slopes=None,
                     cap: float = 0.0, scale=None, out=None, stream=None):
    """Attention of new tokens over the cache (see the module), which holds theirs already:
    q [T, H, D] in bf16 or fp16, Hk dividing H, channels contiguous, token and head strides
    that are multiples of 8 elements and at least D.  Returns ``(out, lse)`` -- out [T, H, D]
    contiguous, lse [H, T] fp32, natural -- or None when not supported.

    ``cu`` as for ``cache_append``; query i of a sequence's n stands at its token lengths[s] -
    n + i and sees the tokens up to its own, or all of its sequence without ``causal``.
    ``cap``, ``slopes`` and ``scale`` as for ``attention_packed``.  page_size is a multiple of 8
    up to 256, D of 16 up to 128.  A query that sees no key, or of no sequence, has out 0 and
    lse -inf."""
    L, T = _start()
    found = _cache_args(k_pages, v_pages, k_scales, v_scales, table, lengths, cu, T)
    if found is None or not isinstance(q, T.Tensor):
        return None
    cache, pool, device = found
    dtype, shape = q.dtype, q.shape
    kind = T.formats.get(dtype)
    if kind not in (0, 1) or _wants_grad(q, slopes) or not _heads_like(q, dtype, device, T):
        return None
    tokens, heads, dim = shape
    scale, cap = 1.0 / math.sqrt(max(1, dim)) if scale is None else scale, cap or 0.0
    if dim != pool[3] or heads > 1024 or not (abs(scale) < 1e38 and abs(cap) < 1e38):
        return None
    if slopes is not None and not (isinstance(slopes, T.Tensor) and slopes.dtype == T.float32 and slopes.device == device
                                   and slopes.shape == (heads,) and slopes.is_contiguous()):
        return None
    if out is not None and not (_like(out, q, T) and out.is_contiguous()):
        return None

    def go(handle):
        o = T.empty(shape, dtype=dtype, device=device) if out is None else out
        lse = T.empty((heads, tokens), dtype=T.float32, device=device)
        need = max(1, L.gn_attn_cached_workspace_bytes(tokens, table.shape[0], heads, pool[2], dim))
        workspace = T.empty(need, dtype=T.uint8, device=device)
        args = _ATTN.pack(q.data_ptr(), o.data_ptr(), lse.data_ptr(), 0 if slopes is None else slopes.data_ptr(),
                          *_head_strides(shape, q.stride()), tokens, scale, cap, heads, bool(causal), kind)
        rc = L.gn_attn_cached(cache, args, workspace.data_ptr(), need, handle)
        return (o, lse) if rc == 0 or _finish(rc, "gn_attn_cached") else None
    return _run(device, stream, (q, k_pages, v_pages, k_scales, v_scales, table, lengths, cu, slopes, out), go)
