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
from .gnsilu import _finish, _grad_blocked, _torch, lib

MAX_AXES = 8


# A call of a small size costs more on the host than on the GPU, so what every
# call asks is looked up once.
@functools.cache
def _formats():
    torch = _torch()
    return {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


@functools.cache
def _position_formats():
    torch = _torch()
    return {torch.int32: 0, torch.int64: 1, torch.float32: 2}


@functools.cache
def _raw_stream():
    """Device index -> the current stream's handle."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _kind(t):
    """The C format of a tensor's dtype, or None."""
    return _formats().get(t.dtype)


def _is_cuda(*ts) -> bool:
    Tensor = _torch().Tensor
    for t in ts:
        if not (isinstance(t, Tensor) and t.is_cuda):
            return False
    return True


def _run(device, stream, inputs, go):
    """``go(handle)`` on `device` and, if one is given, `stream`: what it
    allocates belongs to that stream, and the inputs are kept from being
    reused before the stream is done with them."""
    torch = _torch()
    if stream is None:
        if device.index == torch.cuda.current_device():
            return go(_raw_stream()(device.index))
        with torch.cuda.device(device):
            return go(_raw_stream()(device.index))
    with torch.cuda.device(device), torch.cuda.stream(stream):
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        return go(stream.cuda_stream)


def _lib():
    return gnsilu._lib or lib()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _head_strides(t):
    """Token and head stride; of an axis of length one the packed ones (torch
    leaves it any stride there)."""
    return (t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2],
            t.stride(1) if t.shape[1] > 1 else t.shape[2])


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def gn_layer_norm_workspace_bytes(rows: int, cols: int) -> int:
    return int(_lib().gn_layer_norm_workspace_bytes(rows, cols))


def _rows_of(t):
    """(rows, row stride) of a tensor seen as rows of its contiguous last
    axis with one stride between them, or None if it is not that."""
    cols = t.shape[-1]
    if t.stride(-1) != 1 and cols > 1:
        return None
    rows = t.numel() // cols
    if rows <= 1:
        return rows, cols
    dims = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    for (_, outer), (n, inner) in zip(dims, dims[1:]):
        if outer != n * inner:
            return None
    return (rows, dims[-1][1]) if dims[-1][1] >= cols else None


def _norm_operand(t, like) -> bool:
    return _is_cuda(t) and t.shape == like.shape and t.dtype == like.dtype and t.device == like.device


def _param_ok(t, x, dtype=None) -> bool:
    return (_is_cuda(t) and t.device == x.device and t.dim() == 1 and t.numel() == x.shape[-1] and t.is_contiguous()
            and _kind(t) is not None and (dtype is None or t.dtype == dtype))


def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, out=None, stream=None):
    """Layer norm over the last axis of a bf16, fp16 or fp32 CUDA tensor
    [..., C], C up to 16384: ``(y, mean, rstd)`` with y shaped like x (``out``
    if given; it may be x) and fp32 statistics shaped ``x.shape[:-1]`` for
    ``layer_norm_backward``; None when not supported.

    ``weight`` and ``bias`` (bias only with a weight): contiguous [C] tensors
    of one dtype, any of the three.  x's rows need a contiguous last axis and
    one stride between rows (a column slice of a wider tensor is fine)."""
    L = _lib()
    torch = _torch()
    if not _is_cuda(x) or _kind(x) is None or x.dim() < 1 or x.shape[-1] < 1 or _grad_blocked(x, weight, bias):
        return None
    if bias is not None and weight is None:
        return None
    if weight is not None and not _param_ok(weight, x):
        return None
    if bias is not None and not _param_ok(bias, x, weight.dtype):
        return None
    if out is not None and not _norm_operand(out, x):
        return None
    rx = _rows_of(x)
    ry = rx if out is None and x.is_contiguous() else _rows_of(out) if out is not None else None
    if rx is None or (out is not None and ry is None):
        return None

    def go(handle):
        y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        cols = x.shape[-1]
        rc = L.gn_layer_norm(x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                             rx[0], cols, rx[1], cols if ry is None else ry[1], eps, _kind(x),
                             0 if weight is None else _kind(weight), handle)
        return (y, mean, rstd) if rc == 0 or _finish(rc, "gn_layer_norm") else None
    return _run(x.device, stream, (x, weight, bias, out), go)


def layer_norm_backward(dy, x, mean, rstd, weight=None, out=None, stream=None):
    """Backward pass of ``layer_norm``: ``(dx, dweight, dbias)`` from the
    gradient dy of its output, its input x, the statistics that it returned
    and its weight; dweight and dbias have the weight's dtype and are None
    without one.  dx is ``out`` if given (it may be dy or x).  None when not
    supported."""
    L = _lib()
    torch = _torch()
    if not _is_cuda(x, dy, mean, rstd) or _kind(x) is None or x.dim() < 1 or x.shape[-1] < 1:
        return None
    if not _norm_operand(dy, x) or _grad_blocked(dy, x, weight):
        return None
    for s in (mean, rstd):
        if s.dtype != torch.float32 or s.shape != x.shape[:-1] or not s.is_contiguous() or s.device != x.device:
            return None
    if weight is not None and not _param_ok(weight, x):
        return None
    if out is not None and not _norm_operand(out, x):
        return None
    cols = x.shape[-1]
    rg, rx, ro = _rows_of(dy), _rows_of(x), (None, cols) if out is None else _rows_of(out)
    if rg is None or rx is None or ro is None:
        return None

    def go(handle):
        dx = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = db = workspace = None
        need = 0
        if weight is not None:
            dw, db = torch.empty_like(weight), torch.empty_like(weight)
            need = max(1, L.gn_layer_norm_workspace_bytes(rx[0], cols))
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        rc = L.gn_layer_norm_backward(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(),
                                      dx.data_ptr(), _ptr(dw), _ptr(db), rx[0], cols, rg[1], rx[1], ro[1], _kind(x),
                                      0 if weight is None else _kind(weight), _ptr(workspace), need, handle)
        return (dx, dw, db) if rc == 0 or _finish(rc, "gn_layer_norm_backward") else None
    return _run(x.device, stream, (dy, x, mean, rstd, weight, out), go)


# ---------------------------------------------------------------------------
# rotary positions over several axes
# ---------------------------------------------------------------------------
_Strides = ctypes.c_int64 * 8


@functools.lru_cache(maxsize=64)
def _axes_array(*axes_dim):
    return (ctypes.c_int64 * len(axes_dim))(*axes_dim)


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
    L = _lib()
    torch = _torch()
    ts = [q] if k is None else [q, k]
    if not _is_cuda(*ts, positions) or _grad_blocked(*ts) or _kind(q) is None:
        return None
    axes_dim = [int(n) for n in axes_dim]
    if not 1 <= len(axes_dim) <= MAX_AXES:
        return None
    if positions.dim() != 2 or positions.shape[1] != len(axes_dim) or not positions.is_contiguous() \
            or _position_formats().get(positions.dtype) is None or positions.device != q.device:
        return None
    for t in ts:
        if t.dim() != 3 or t.dtype != q.dtype or t.device != q.device or t.shape[0] != positions.shape[0] \
                or t.shape[2] != q.shape[2] or (t.shape[2] > 1 and t.stride(2) != 1) or t.shape[1] < 1:
            return None
    if out is not None:
        if len(out) != 2 or (k is None) != (out[1] is None):
            return None
        for t, o in zip(ts, out):
            if not (_is_cuda(o) and o.shape == t.shape and o.dtype == t.dtype and o.device == t.device
                    and (o.shape[2] <= 1 or o.stride(2) == 1)):
                return None

    def go(handle):
        outs = out if out is not None else [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in ts]
        strides = [0] * 8
        for n, t in enumerate(ts):
            strides[2 * n:2 * n + 2] = _head_strides(t)
            strides[4 + 2 * n:6 + 2 * n] = _head_strides(outs[n])
        rc = L.gn_rope_nd(q.data_ptr(), _ptr(k), outs[0].data_ptr(), None if k is None else outs[1].data_ptr(),
                          _Strides(*strides), q.shape[0], q.shape[1], 0 if k is None else k.shape[1], q.shape[2],
                          positions.data_ptr(), _position_formats()[positions.dtype], len(axes_dim), _axes_array(*axes_dim),
                          theta, bool(interleaved), bool(inverse), _kind(q), handle)
        return (outs[0], None if k is None else outs[1]) if rc == 0 or _finish(rc, "gn_rope_nd") else None
    return _run(q.device, stream, (*ts, positions, *(out or ())), go)


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
    return int(_lib().gn_attn_packed_workspace_bytes(tokens_q, heads))


def _heads_ok(t, like=None) -> bool:
    return (_is_cuda(t) and t.dim() == 3 and _kind(t) in (0, 1) and (t.shape[2] <= 1 or t.stride(2) == 1)
            and (like is None or (t.dtype == like.dtype and t.device == like.device and t.shape[2] == like.shape[2])))


def _packed_args(q, k, v, cu_q, cu_k, causal, prefix, slopes, cap, scale):
    """The C arguments without the outputs, or None if not supported."""
    torch = _torch()
    if not (_heads_ok(q) and _heads_ok(k, q) and _heads_ok(v, q)) or k.shape != v.shape or _grad_blocked(q, k, v):
        return None
    if q.shape[1] < 1 or k.shape[1] < 1 or q.shape[1] % k.shape[1]:
        return None
    docs = 1
    if (cu_q is None) != (cu_k is None):
        return None
    if cu_q is not None:
        for t in (cu_q, cu_k):
            if not (_is_cuda(t) and t.dtype == torch.int32 and t.dim() == 1 and t.is_contiguous()
                    and t.device == q.device and t.numel() == cu_q.numel() and t.numel() >= 2):
                return None
        docs = cu_q.numel() - 1
    if prefix is not None and not (causal and _is_cuda(prefix) and prefix.dtype == torch.int32
                                   and prefix.shape == (docs,) and prefix.is_contiguous()
                                   and prefix.device == q.device):
        return None
    if slopes is not None and not (_is_cuda(slopes) and slopes.dtype == torch.float32
                                   and slopes.shape == (q.shape[1],) and slopes.is_contiguous()
                                   and slopes.device == q.device) or _grad_blocked(slopes):
        return None
    a = PackedAttnArgs()
    for name, t in (("q", q), ("k", k), ("v", v)):
        setattr(a, name, _ptr(t))
        token, head = _head_strides(t)
        setattr(a, name + "_token", token)
        setattr(a, name + "_head", head)
    a.tokens_q, a.tokens_k = q.shape[0], k.shape[0]
    a.cu_q, a.cu_k, a.prefix, a.slopes = _ptr(cu_q), _ptr(cu_k), _ptr(prefix), _ptr(slopes)
    a.scale = 1.0 / math.sqrt(max(1, q.shape[2])) if scale is None else float(scale)
    a.cap = float(cap or 0.0)
    a.heads, a.kv_heads, a.dim, a.docs = q.shape[1], k.shape[1], q.shape[2], docs
    a.causal, a.format = int(bool(causal)), _kind(q)
    return a


def attention_packed(q, k, v, cu_q=None, cu_k=None, causal: bool = False, prefix=None, slopes=None, cap: float = 0.0,
                     scale=None, out=None, stream=None):
    """Attention of documents packed one after the other along the token axis
    (images of several sizes with their texts, prompts, new tokens beside a
    cache): q [Tq, H, D], k and v [Tk, Hk, D] in bf16 or fp16, Hk dividing H,
    D a multiple of 8 up to 128, any token and head strides that are multiples
    of 8 elements.  Returns ``(out, lse)`` -- out [Tq, H, D] contiguous, lse
    [H, Tq] fp32, natural -- or None when not supported.

    ``cu_q`` and ``cu_k`` (int32 [docs + 1], on the GPU) hold where each
    document's queries and keys begin; both None: one document of everything.
    A document's last query stands at its last key, so one query for each
    document is a decode step.  A query sees its document's keys: all of them,
    or with ``causal`` those up to its own position and the first
    ``prefix[d]`` (int32 [docs]).  ``cap``: scores are bent to cap tanh(t /
    cap).  ``slopes`` (fp32 [H]): slopes[h] times the distance of the two
    positions is taken off.  ``scale``: 1 / sqrt(D) if None.  A query that sees
    no key has out 0 and lse -inf."""
    L = _lib()
    torch = _torch()
    a = _packed_args(q, k, v, cu_q, cu_k, causal, prefix, slopes, cap, scale)
    if a is None:
        return None
    if out is not None and not (_is_cuda(out) and out.shape == q.shape and out.dtype == q.dtype
                                and out.device == q.device and out.is_contiguous()):
        return None

    def go(handle):
        o = out if out is not None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
        a.out, a.lse = o.data_ptr(), lse.data_ptr()
        rc = L.gn_attn_packed(ctypes.byref(a), handle)
        return (o, lse) if rc == 0 or _finish(rc, "gn_attn_packed") else None
    return _run(q.device, stream, (q, k, v, cu_q, cu_k, prefix, slopes, out), go)


def attention_packed_backward(dout, q, k, v, out, lse, cu_q=None, cu_k=None, causal: bool = False, prefix=None,
                              slopes=None, cap: float = 0.0, scale=None, stream=None):
    """Backward pass of ``attention_packed``: ``(dq, dk, dv)``, contiguous and
    shaped like q, k and v, from the gradient dout of its output (any strides
    that are multiples of 8 elements), its inputs and what it returned; the
    remaining arguments as for the forward call.  dk and dv are summed over
    the query heads that share a key / value head.  The slopes have no
    gradient.  None when not supported."""
    L = _lib()
    torch = _torch()
    a = _packed_args(q, k, v, cu_q, cu_k, causal, prefix, slopes, cap, scale)
    if a is None or not _heads_ok(dout, q) or dout.shape != q.shape or _grad_blocked(dout, out, lse):
        return None
    if not (_is_cuda(out, lse) and out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous()
            and out.device == q.device and lse.shape == (q.shape[1], q.shape[0]) and lse.dtype == torch.float32
            and lse.is_contiguous() and lse.device == q.device):
        return None
    a.out, a.lse = _ptr(out), _ptr(lse)

    def go(handle):
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        need = max(1, L.gn_attn_packed_workspace_bytes(q.shape[0], q.shape[1]))
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        rc = L.gn_attn_packed_backward(ctypes.byref(a), dout.data_ptr(), *_head_strides(dout), dq.data_ptr(),
                                       dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), need, handle)
        return (dq, dk, dv) if rc == 0 or _finish(rc, "gn_attn_packed_backward") else None
    return _run(q.device, stream, (dout, q, k, v, out, lse, cu_q, cu_k, prefix, slopes), go)
