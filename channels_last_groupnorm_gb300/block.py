"""Python binding of the transformer-block operators of libgnsilu
(``include/gnsilu.h``): layer norm and its backward pass, rotary positions
over several axes, and attention of packed documents with its backward pass.

As in ``gnsilu``, every step runs in the library's kernels; this module checks
tensor metadata, allocates outputs and workspaces and calls the C entry point.
Unsupported input (not CUDA, a dtype, width, layout or alignment the library
does not take, or a tensor that requires grad while gradients are recorded)
gives ``None``, so that callers can fall back to their own path; a CUDA or
kernel failure raises ``GnError``.  The backward passes are calls of their own:
a caller's ``torch.autograd.Function`` saves what they need.

``stream``: a ``torch.cuda.Stream`` to run on instead of the current one.
Outputs and workspaces are allocated for it, and the inputs are recorded on
it; ordering it after the work that produces the inputs is up to the caller,
as everywhere in torch.
"""
from __future__ import annotations

import ctypes
import functools
import math

from . import gnsilu
from .gnsilu import _finish, lib

MAX_AXES = 8


# A call of a small size costs more on the host than on the GPU, so what every
# call asks is looked up once, and a tensor's shape and strides are asked for
# once each.
class _Torch:
    """torch, its tensor type and what the entry points need of it, from the
    first call on."""
    ready = False

    @classmethod
    def load(cls):
        import torch
        cls.torch, cls.Tensor, cls.empty = torch, torch.Tensor, torch.empty
        cls.formats = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
        cls.positions = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
        cls.float32, cls.int32, cls.uint8 = torch.float32, torch.int32, torch.uint8
        cls.recording = staticmethod(torch.is_grad_enabled)
        cls.current = staticmethod(torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.handle = staticmethod(raw or (lambda index: torch.cuda.current_stream(index).cuda_stream))
        cls.ready = True


def _start():
    """(The library, torch's parts)."""
    if not _Torch.ready:
        _Torch.load()
    return gnsilu._lib or lib(), _Torch


def _wants_grad(*ts) -> bool:
    if _Torch.recording():
        for t in ts:
            if t is not None and t.requires_grad:
                return True
    return False


def _run(device, stream, inputs, go):
    """``go(handle)`` on `device` and, if one is given, `stream`: what it
    allocates belongs to that stream, and the inputs are kept from being
    reused before the stream is done with them."""
    T = _Torch
    if stream is None:
        index = device.index
        if index == T.current():
            return go(T.handle(index))
        with T.torch.cuda.device(device):
            return go(T.handle(index))
    with T.torch.cuda.device(device), T.torch.cuda.stream(stream):
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        return go(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _head_strides(shape, strides):
    """Token and head stride; of an axis of length one the packed ones (torch
    leaves it any stride there)."""
    return (strides[0] if shape[0] > 1 else shape[1] * shape[2], strides[1] if shape[1] > 1 else shape[2])


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def gn_layer_norm_workspace_bytes(rows: int, cols: int) -> int:
    return int(_start()[0].gn_layer_norm_workspace_bytes(rows, cols))


def _flat_stride(dims, alone):
    """The one stride of axes [(length, stride), ...] (0 of a broadcast one;
    `alone` where every axis has length one), or None."""
    dims = [(n, s) for n, s in dims if n != 1]
    for (_, outer), (n, inner) in zip(dims, dims[1:]):
        if outer != n * inner:
            return None
    return dims[-1][1] if dims else alone


def _row_strides(shape, all_strides):
    """(inner, (outer, stride) of each tensor, ...) of the rows of tensors of
    one shape with contiguous last axes: inner 0 where every one has a single
    stride between its rows, else the last but one axis' length.  None if the
    rows have no such strides."""
    cols = shape[-1]
    lead, found = shape[:-1], []
    for strides in all_strides:
        if strides[-1] != 1 and cols > 1:
            return None
        stride = strides[0] if len(lead) == 1 and lead[0] != 1 else _flat_stride(list(zip(lead, strides)), cols)
        if stride is None:
            break
        found += [0, stride]
    else:
        return 0, found
    if len(lead) < 2:
        return None
    found = []
    for strides in all_strides:
        outer = _flat_stride(list(zip(lead[:-1], strides)), 0)
        if outer is None:
            return None
        found += [outer, strides[-2] if lead[-1] > 1 else cols]
    return lead[-1], found


_Strides4, _Strides6 = ctypes.c_int64 * 4, ctypes.c_int64 * 6


def _packed_strides(shape):
    strides = [1]
    for n in shape[:0:-1]:
        strides.insert(0, strides[0] * n)
    return strides


def _like(t, x, T) -> bool:
    return isinstance(t, T.Tensor) and t.shape == x.shape and t.dtype == x.dtype and t.device == x.device


def _param_format(t, cols, device, T):
    """The format of a weight or bias vector, or None."""
    if not (isinstance(t, T.Tensor) and t.device == device and t.dim() == 1 and t.numel() == cols and t.is_contiguous()):
        return None
    return T.formats.get(t.dtype)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, out=None, stream=None):
    """Layer norm over the last axis of a bf16, fp16 or fp32 CUDA tensor
    [..., C], C up to 16384: ``(y, mean, rstd)`` with y shaped like x (``out``
    if given; it may be x) and fp32 statistics shaped ``x.shape[:-1]`` for
    ``layer_norm_backward``; None when not supported.

    ``weight`` and ``bias`` (bias only with a weight): contiguous [C] tensors
    of one dtype, any of the three.  x needs a contiguous last axis and one or
    two strides between its rows: a column slice of a wider tensor is fine, and
    so are some heads [T, H, C] of a fused projection, and rows broadcast by
    ``expand`` (``out`` must have rows of its own)."""
    L, T = _start()
    if not (isinstance(x, T.Tensor) and x.is_cuda):
        return None
    shape, device, kind = x.shape, x.device, T.formats.get(x.dtype)
    if kind is None or not shape or shape[-1] < 1 or _wants_grad(x, weight, bias):
        return None
    cols, wkind = shape[-1], 0
    if weight is not None:
        wkind = _param_format(weight, cols, device, T)
        if wkind is None or (bias is not None and _param_format(bias, cols, device, T) != wkind):
            return None
    elif bias is not None:
        return None
    if out is not None and not _like(out, x, T):
        return None
    if out is None and x.is_contiguous():
        inner, strides = 0, (0, cols, 0, cols)
    else:
        y_strides = _packed_strides(shape) if out is None else out.stride()
        rows_at = _row_strides(shape, (x.stride(), y_strides))
        if rows_at is None:
            return None
        inner, strides = rows_at

    def go(handle):
        y = T.empty(shape, dtype=x.dtype, device=device) if out is None else out
        mean = T.empty(shape[:-1], dtype=T.float32, device=device)
        rstd = T.empty(shape[:-1], dtype=T.float32, device=device)
        rc = L.gn_layer_norm(x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                             mean.numel(), cols, inner or max(1, mean.numel()), _Strides4(*strides), eps, kind, wkind, handle)
        return (y, mean, rstd) if rc == 0 or _finish(rc, "gn_layer_norm") else None
    return _run(device, stream, (x, weight, bias, out), go)


def layer_norm_backward(dy, x, mean, rstd, weight=None, out=None, stream=None):
    """Backward pass of ``layer_norm``: ``(dx, dweight, dbias)`` from the
    gradient dy of its output, its input x, the statistics that it returned
    and its weight; dweight and dbias have the weight's dtype and are None
    without one.  dy may be broadcast over rows, as the gradient of a sum over
    tokens is.  dx is ``out`` if given (it may be dy or x).  None when not
    supported."""
    L, T = _start()
    if not (isinstance(x, T.Tensor) and x.is_cuda):
        return None
    shape, device, kind = x.shape, x.device, T.formats.get(x.dtype)
    if kind is None or not shape or shape[-1] < 1 or not _like(dy, x, T) or _wants_grad(dy, x, weight):
        return None
    for s in (mean, rstd):
        if not (isinstance(s, T.Tensor) and s.dtype == T.float32 and s.shape == shape[:-1] and s.is_contiguous()
                and s.device == device):
            return None
    cols, wkind = shape[-1], 0
    if weight is not None:
        wkind = _param_format(weight, cols, device, T)
        if wkind is None:
            return None
    if out is not None and not _like(out, x, T):
        return None
    if out is None and x.is_contiguous() and dy.is_contiguous():
        inner, strides = 0, (0, cols, 0, cols, 0, cols)
    else:
        rows_at = _row_strides(shape, (dy.stride(), x.stride(), _packed_strides(shape) if out is None else out.stride()))
        if rows_at is None:
            return None
        inner, strides = rows_at

    def go(handle):
        dx = T.empty(shape, dtype=x.dtype, device=device) if out is None else out
        rows = mean.numel()
        dw = db = workspace = None
        need = 0
        if weight is not None:
            dw, db = T.torch.empty_like(weight), T.torch.empty_like(weight)
            need = max(1, L.gn_layer_norm_workspace_bytes(rows, cols))
            workspace = T.empty(need, dtype=T.uint8, device=device)
        rc = L.gn_layer_norm_backward(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(),
                                      dx.data_ptr(), _ptr(dw), _ptr(db), rows, cols, inner or max(1, rows), _Strides6(*strides),
                                      kind, wkind,
                                      _ptr(workspace), need, handle)
        return (dx, dw, db) if rc == 0 or _finish(rc, "gn_layer_norm_backward") else None
    return _run(device, stream, (dy, x, mean, rstd, weight, out), go)


# ---------------------------------------------------------------------------
# rotary positions over several axes
# ---------------------------------------------------------------------------
_Strides = ctypes.c_int64 * 8


@functools.lru_cache(maxsize=64)
def _axes_array(axes_dim):
    return (ctypes.c_int64 * len(axes_dim))(*axes_dim)


def _heads_like(t, dtype, device, T) -> bool:
    """[tokens, heads, channels] with contiguous channels."""
    return (isinstance(t, T.Tensor) and t.dtype == dtype and t.device == device and t.dim() == 3 and t.shape[1] >= 1
            and (t.stride(2) == 1 or t.shape[2] <= 1))


def rope_nd(q, k, positions, axes_dim, theta: float = 10000.0, interleaved: bool = True, inverse: bool = False,
            out=None, stream=None):
    """Rotary positions over several axes (time, height, width, ...) of the
    query heads q [T, H, D] and the key heads k [T, Hk, D] (or None), bf16,
    fp16 or fp32 with contiguous channels: ``(q_out, k_out)``, or None when
    not supported.

    ``positions`` [T, axes] (int32, int64 or fp32) hold every token's place on
    each axis; ``axes_dim`` says how many channels of a head turn with each
    axis (even numbers; channels past their sum pass unchanged).  Pair i of an
    axis with d channels turns by ``position * theta ** (-2 i / d)``; a pair is
    two neighbours if ``interleaved``, else channel p of either half of the
    turned channels.  ``inverse`` turns back: applied to the outputs'
    gradients it gives the inputs'.  ``out``: a pair of tensors for the
    results, which may be q and k themselves."""
    L, T = _start()
    if not (isinstance(q, T.Tensor) and q.is_cuda and isinstance(positions, T.Tensor)):
        return None
    dtype, device = q.dtype, q.device
    kind, place, axes_dim = T.formats.get(dtype), T.positions.get(positions.dtype), tuple(axes_dim)
    ts = (q,) if k is None else (q, k)
    if kind is None or place is None or _wants_grad(*ts) or not 1 <= len(axes_dim) <= MAX_AXES:
        return None
    if positions.shape != (q.shape[0], len(axes_dim)) or positions.device != device or not positions.is_contiguous():
        return None
    shapes, strides = [], []
    for t in ts:
        if not _heads_like(t, dtype, device, T):
            return None
        shapes.append(t.shape)
        strides.append(_head_strides(shapes[-1], t.stride()))
    if k is not None and (shapes[1][0] != shapes[0][0] or shapes[1][2] != shapes[0][2]):
        return None
    if out is not None:
        if len(out) != 2 or (k is None) != (out[1] is None):
            return None
        for shape, o in zip(shapes, out):
            if not _heads_like(o, dtype, device, T) or o.shape != shape:
                return None

    def go(handle):
        outs = [T.empty(s, dtype=dtype, device=device) for s in shapes] if out is None else out
        to = [(s[1] * s[2], s[2]) if out is None else _head_strides(s, o.stride()) for s, o in zip(shapes, outs)]
        tokens, heads, dim = shapes[0]
        if k is None:
            rc = L.gn_rope_nd(q.data_ptr(), None, outs[0].data_ptr(), None, _Strides(*strides[0], 0, 0, *to[0], 0, 0),
                              tokens, heads, 0, dim, positions.data_ptr(), place, len(axes_dim), _axes_array(axes_dim),
                              theta, bool(interleaved), bool(inverse), kind, handle)
        else:
            rc = L.gn_rope_nd(q.data_ptr(), k.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(),
                              _Strides(*strides[0], *strides[1], *to[0], *to[1]), tokens, heads, shapes[1][1], dim,
                              positions.data_ptr(), place, len(axes_dim), _axes_array(axes_dim), theta,
                              bool(interleaved), bool(inverse), kind, handle)
        return (outs[0], None if k is None else outs[1]) if rc == 0 or _finish(rc, "gn_rope_nd") else None
    return _run(device, stream, (*ts, positions, *(out or ())), go)


# ---------------------------------------------------------------------------
# attention of packed documents
# ---------------------------------------------------------------------------
class PackedAttnArgs(ctypes.Structure):
    """``gn_attn_packed_args`` of include/gnsilu.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "lse")]
                + [(n, ctypes.c_int64) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head",
                                                 "tokens_q", "tokens_k")]
                + [(n, ctypes.c_void_p) for n in ("cu_q", "cu_k", "prefix", "slopes")]
                + [(n, ctypes.c_float) for n in ("scale", "cap")]
                + [(n, ctypes.c_int) for n in ("heads", "kv_heads", "dim", "docs", "causal", "format")])


def gn_attn_packed_workspace_bytes(tokens_q: int, heads: int) -> int:
    return int(_start()[0].gn_attn_packed_workspace_bytes(tokens_q, heads))


def _ends_like(t, docs, device, T) -> bool:
    return (isinstance(t, T.Tensor) and t.dtype == T.int32 and t.device == device and t.dim() == 1
            and t.numel() == docs and t.is_contiguous())


def _packed_args(q, k, v, cu_q, cu_k, causal, prefix, slopes, cap, scale, T):
    """The C arguments without the outputs, or None if not supported."""
    if not (isinstance(q, T.Tensor) and q.is_cuda):
        return None
    dtype, device = q.dtype, q.device
    kind = T.formats.get(dtype)
    if kind not in (0, 1) or _wants_grad(q, k, v, slopes):
        return None
    for t in (q, k, v):
        if not _heads_like(t, dtype, device, T):
            return None
    shape, kv_shape = q.shape, k.shape
    tokens, heads, dim = shape
    if v.shape != kv_shape or kv_shape[2] != dim or heads % kv_shape[1]:
        return None
    docs = 1
    if cu_q is None:
        if cu_k is not None:
            return None
    else:
        if not isinstance(cu_q, T.Tensor):
            return None
        docs = cu_q.numel() - 1
        if docs < 1 or not _ends_like(cu_q, docs + 1, device, T) or not _ends_like(cu_k, docs + 1, device, T):
            return None
    if prefix is not None and not (causal and _ends_like(prefix, docs, device, T)):
        return None
    if slopes is not None and not (isinstance(slopes, T.Tensor) and slopes.dtype == T.float32 and slopes.device == device
                                   and slopes.shape == (heads,) and slopes.is_contiguous()):
        return None
    # (in the order of the structure; the outputs come later)
    return PackedAttnArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, *_head_strides(shape, q.stride()),
                          *_head_strides(kv_shape, k.stride()), *_head_strides(kv_shape, v.stride()), tokens, kv_shape[0],
                          _ptr(cu_q), _ptr(cu_k), _ptr(prefix), _ptr(slopes),
                          1.0 / math.sqrt(max(1, dim)) if scale is None else scale, cap or 0.0, heads, kv_shape[1], dim,
                          docs, bool(causal), kind)


def attention_packed(q, k, v, cu_q=None, cu_k=None, causal: bool = False, prefix=None, slopes=None, cap: float = 0.0,
                     scale=None, out=None, stream=None):
    """Attention of documents packed one after the other along the token axis
    (images of several sizes with their texts, prompts, new tokens beside a
    cache): q [Tq, H, D], k and v [Tk, Hk, D] in bf16 or fp16, Hk dividing H,
    D a multiple of 8 up to 128, any token and head strides that are multiples
    of 8 elements and at least D.  Returns ``(out, lse)`` -- out [Tq, H, D] contiguous, lse
    [H, Tq] fp32, natural -- or None when not supported.

    ``cu_q`` and ``cu_k`` (int32 [docs + 1], on the GPU) hold where each
    document's queries and keys begin; both None: one document of everything.
    A document's last query stands at its last key, so one query for each
    document is a decode step; room behind a cache's documents is told by
    documents without queries (cu_q 0 1 1 2 2 ..., cu_k 0 end begin end ...).
    A query sees its document's keys: all of them,
    or with ``causal`` those up to its own position and the first
    ``prefix[d]`` (int32 [docs]).  ``cap``: scores are bent to cap tanh(t /
    cap).  ``slopes`` (fp32 [H]): slopes[h] times the distance of the two
    positions is taken off.  ``scale``: 1 / sqrt(D) if None.  A query that sees
    no key has out 0 and lse -inf."""
    L, T = _start()
    a = _packed_args(q, k, v, cu_q, cu_k, causal, prefix, slopes, cap, scale, T)
    if a is None or (out is not None and not (_like(out, q, T) and out.is_contiguous())):
        return None
    shape, device = q.shape, q.device

    def go(handle):
        o = T.empty(shape, dtype=q.dtype, device=device) if out is None else out
        lse = T.empty((shape[1], shape[0]), dtype=T.float32, device=device)
        a.out, a.lse = o.data_ptr(), lse.data_ptr()
        rc = L.gn_attn_packed(ctypes.byref(a), handle)
        return (o, lse) if rc == 0 or _finish(rc, "gn_attn_packed") else None
    return _run(device, stream, (q, k, v, cu_q, cu_k, prefix, slopes, out), go)


def attention_packed_backward(dout, q, k, v, out, lse, cu_q=None, cu_k=None, causal: bool = False, prefix=None,
                              slopes=None, cap: float = 0.0, scale=None, stream=None):
    """Backward pass of ``attention_packed``: ``(dq, dk, dv)``, contiguous and
    shaped like q, k and v, from the gradient dout of its output (strides as
    for q), its inputs and what it returned; the remaining arguments as for the
    forward call.  In fp16, scale the loss so that dout is not far below 1.  dk and dv are summed over
    the query heads that share a key / value head.  The slopes have no
    gradient.  None when not supported."""
    L, T = _start()
    a = _packed_args(q, k, v, cu_q, cu_k, causal, prefix, slopes, cap, scale, T)
    if a is None or not _like(dout, q, T) or not _heads_like(dout, q.dtype, q.device, T) or _wants_grad(dout, out, lse):
        return None
    shape, device = q.shape, q.device
    if not (_like(out, q, T) and out.is_contiguous() and isinstance(lse, T.Tensor) and lse.device == device
            and lse.shape == (shape[1], shape[0]) and lse.dtype == T.float32 and lse.is_contiguous()):
        return None
    a.out, a.lse = out.data_ptr(), lse.data_ptr()

    def go(handle):
        dq, dk, dv = (T.empty(t.shape, dtype=t.dtype, device=device) for t in (q, k, v))
        need = max(1, L.gn_attn_packed_workspace_bytes(shape[0], shape[1]))
        workspace = T.empty(need, dtype=T.uint8, device=device)
        rc = L.gn_attn_packed_backward(ctypes.byref(a), dout.data_ptr(), *_head_strides(shape, dout.stride()),
                                       dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), need, handle)
        return (dq, dk, dv) if rc == 0 or _finish(rc, "gn_attn_packed_backward") else None
    return _run(device, stream, (dout, q, k, v, out, lse, cu_q, cu_k, prefix, slopes), go)
