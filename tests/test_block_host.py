"""The transformer-block entry points on the host, without a GPU: every kind
of unsupported input is refused with its status before any CUDA call, and the
binding returns None for tensors it does not take.  The 64-bit references
that the GPU tests use are checked against differences here."""
import ctypes
import math

import pytest
import torch

from channels_last_groupnorm_gb300 import block
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from tests import block_ref as br

# stand-in device addresses, far apart (never dereferenced: every call below is refused first)
A, B, C, D, E, F, G, H = (0x1000000000 * n for n in range(1, 9))
S = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    gnbuild.build()


def norm(**kw):
    a = dict(x=A, w=B, b=C, y=D, mean=E, rstd=F, rows=16, cols=64, xs=64, ys=64, eps=1e-6, fmt=0, wfmt=2)
    a.update(kw)
    strides = (ctypes.c_int64 * 4)(a.get("xo", 0), a["xs"], a.get("yo", 0), a["ys"])
    return gs.lib().gn_layer_norm(a["x"], a["w"], a["b"], a["y"], a["mean"], a["rstd"], a["rows"], a["cols"],
                                  a.get("inner", 1 << 40), strides, a["eps"], a["fmt"], a["wfmt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), gs.GN_ERR_NULL), (dict(y=None), gs.GN_ERR_NULL), (dict(w=None), gs.GN_ERR_NULL),
    (dict(fmt=3), gs.GN_ERR_FORMAT), (dict(fmt=-1), gs.GN_ERR_FORMAT), (dict(wfmt=7), gs.GN_ERR_FORMAT),
    (dict(rows=-1), gs.GN_ERR_SHAPE), (dict(cols=0), gs.GN_ERR_CHANNELS), (dict(cols=16385, xs=S, ys=S), gs.GN_ERR_CHANNELS),
    (dict(xs=63), gs.GN_ERR_SHAPE), (dict(ys=0), gs.GN_ERR_SHAPE), (dict(rows=1 << 60), gs.GN_ERR_SHAPE),
    (dict(xs=1 << 62), gs.GN_ERR_SHAPE),
    (dict(inner=0), gs.GN_ERR_SHAPE), (dict(inner=4, xo=100, yo=256), gs.GN_ERR_SHAPE),
    (dict(inner=4, xo=256, yo=255), gs.GN_ERR_SHAPE), (dict(inner=4, rows=1 << 33, xo=256, yo=256), gs.GN_ERR_SHAPE),
    (dict(inner=4, xo=512, yo=512, y=A + 256), gs.GN_ERR_ALIAS),
    (dict(eps=math.nan), gs.GN_ERR_EPS), (dict(eps=-1.0), gs.GN_ERR_EPS), (dict(eps=math.inf), gs.GN_ERR_EPS),
    (dict(x=A + 1), gs.GN_ERR_ALIGN), (dict(y=D + 1), gs.GN_ERR_ALIGN), (dict(w=B + 2), gs.GN_ERR_ALIGN),
    (dict(mean=E + 2), gs.GN_ERR_ALIGN), (dict(fmt=2, x=A + 2), gs.GN_ERR_ALIGN),
    (dict(y=A + 128), gs.GN_ERR_ALIAS), (dict(y=A, ys=128), gs.GN_ERR_ALIAS), (dict(mean=A), gs.GN_ERR_ALIAS),
    (dict(rstd=E + 4), gs.GN_ERR_ALIAS), (dict(w=D), gs.GN_ERR_ALIAS), (dict(b=E), gs.GN_ERR_ALIAS),
])
def test_layer_norm_refuses(kw, code):
    assert norm(**kw) == code


def norm_grad(**kw):
    a = dict(dy=A, x=B, w=C, mean=D, rstd=E, dx=F, dw=G, db=G + S, rows=16, cols=64, gs=64, xs=64, ds=64, fmt=0, wfmt=2,
             ws=H, wsb=1 << 30)
    a.update(kw)
    return gs.lib().gn_layer_norm_backward(a["dy"], a["x"], a["w"], a["mean"], a["rstd"], a["dx"], a["dw"], a["db"],
                                           a["rows"], a["cols"], a.get("inner", 1 << 40),
                                           (ctypes.c_int64 * 6)(0, a["gs"], 0, a["xs"], 0, a["ds"]), a["fmt"], a["wfmt"],
                                           a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), gs.GN_ERR_NULL), (dict(mean=None), gs.GN_ERR_NULL), (dict(dx=None), gs.GN_ERR_NULL),
    (dict(dw=None), gs.GN_ERR_NULL), (dict(w=None), gs.GN_ERR_NULL), (dict(ws=None), gs.GN_ERR_NULL),
    (dict(fmt=5), gs.GN_ERR_FORMAT), (dict(rows=-2), gs.GN_ERR_SHAPE), (dict(cols=0), gs.GN_ERR_CHANNELS),
    (dict(gs=1), gs.GN_ERR_SHAPE), (dict(ds=1), gs.GN_ERR_SHAPE), (dict(ws=H + 16), gs.GN_ERR_ALIGN),
    (dict(rstd=E + 1), gs.GN_ERR_ALIGN), (dict(dx=A + 2), gs.GN_ERR_ALIAS), (dict(dx=B + 2), gs.GN_ERR_ALIAS),
    (dict(db=G), gs.GN_ERR_ALIAS), (dict(ws=A), gs.GN_ERR_ALIAS), (dict(dw=D), gs.GN_ERR_ALIAS),
])
def test_layer_norm_backward_refuses(kw, code):
    assert norm_grad(**kw) == code


def rope(**kw):
    a = dict(q=A, k=B, qo=C, ko=D, strides=[512, 128, 128, 128, 512, 128, 128, 128], tokens=8, heads=4, kv=1, dim=128,
             pos=E, pfmt=0, axes=[32, 96], theta=1e4, fmt=0)
    a.update(kw)
    st = None if a["strides"] is None else (ctypes.c_int64 * 8)(*a["strides"])
    ax = (ctypes.c_int64 * max(1, len(a["axes"])))(*a["axes"])
    return gs.lib().gn_rope_nd(a["q"], a["k"], a["qo"], a["ko"], st, a["tokens"], a["heads"], a["kv"], a["dim"], a["pos"],
                               a["pfmt"], len(a["axes"]), ax, a["theta"], 1, 0, a["fmt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), gs.GN_ERR_NULL), (dict(ko=None), gs.GN_ERR_NULL), (dict(k=None, ko=None), gs.GN_ERR_NULL),
    (dict(pos=None), gs.GN_ERR_NULL), (dict(strides=None), gs.GN_ERR_NULL),
    (dict(fmt=3), gs.GN_ERR_FORMAT), (dict(pfmt=3), gs.GN_ERR_FORMAT),
    (dict(tokens=-1), gs.GN_ERR_SHAPE), (dict(heads=0), gs.GN_ERR_SHAPE),
    (dict(strides=[512, 128, 128, 128, 64, 128, 128, 128]), gs.GN_ERR_SHAPE),
    (dict(axes=[]), gs.GN_ERR_CHANNELS), (dict(axes=[2] * 9), gs.GN_ERR_CHANNELS), (dict(axes=[31, 33]), gs.GN_ERR_CHANNELS),
    (dict(axes=[130]), gs.GN_ERR_CHANNELS), (dict(axes=[0, 64]), gs.GN_ERR_CHANNELS), (dict(dim=1), gs.GN_ERR_CHANNELS),
    (dict(theta=0.0), gs.GN_ERR_EPS), (dict(theta=math.nan), gs.GN_ERR_EPS),
    (dict(q=A + 1), gs.GN_ERR_ALIGN), (dict(pos=E + 2), gs.GN_ERR_ALIGN),
    (dict(qo=A + 256), gs.GN_ERR_ALIAS), (dict(qo=B), gs.GN_ERR_ALIAS), (dict(ko=C), gs.GN_ERR_ALIAS), (dict(qo=E), gs.GN_ERR_ALIAS),
])
def test_rope_refuses(kw, code):
    assert rope(**kw) == code


def attn(dim=64, heads=4, kv=2, tq=100, tk=200, backward=False, **kw):
    a = block.PackedAttnArgs()
    d = dict(q=A, k=B, v=C, out=D, lse=E, q_token=heads * dim, q_head=dim, k_token=kv * dim, k_head=dim, v_token=kv * dim,
             v_head=dim, tokens_q=tq, tokens_k=tk, cu_q=F, cu_k=F + S, prefix=None, slopes=None, scale=0.1, cap=0.0,
             heads=heads, kv_heads=kv, dim=dim, docs=3, causal=0, format=0)
    extra = dict(dout=G, dt=heads * dim, dh=dim, dq=H, dk=H + 64 * S, dv=H + 128 * S, ws=H + 256 * S, wsb=1 << 20)
    for n, v in kw.items():
        (d if n in d else extra)[n] = v
    for n, v in d.items():
        setattr(a, n, v)
    if not backward:
        return gs.lib().gn_attn_packed(ctypes.byref(a), None)
    return gs.lib().gn_attn_packed_backward(ctypes.byref(a), extra["dout"], extra["dt"], extra["dh"], extra["dq"],
                                            extra["dk"], extra["dv"], extra["ws"], extra["wsb"], None)


BAD = [
    (dict(q=None), gs.GN_ERR_NULL), (dict(v=None), gs.GN_ERR_NULL), (dict(lse=None), gs.GN_ERR_NULL),
    (dict(cu_q=None), gs.GN_ERR_NULL), (dict(format=2), gs.GN_ERR_FORMAT), (dict(tokens_q=-1), gs.GN_ERR_SHAPE),
    (dict(tokens_k=(1 << 30) + 1), gs.GN_ERR_SHAPE), (dict(docs=0), gs.GN_ERR_SHAPE), (dict(q_token=-256), gs.GN_ERR_SHAPE),
    (dict(k_token=0), gs.GN_ERR_SHAPE), (dict(v_head=8), gs.GN_ERR_SHAPE), (dict(heads=3), gs.GN_ERR_CHANNELS),
    (dict(kv_heads=0), gs.GN_ERR_CHANNELS), (dict(dim=136), gs.GN_ERR_CHANNELS), (dict(dim=20), gs.GN_ERR_CHANNELS),
    (dict(scale=math.inf), gs.GN_ERR_EPS), (dict(cap=-1.0), gs.GN_ERR_EPS), (dict(cap=math.nan), gs.GN_ERR_EPS),
    (dict(prefix=F + 2 * S), gs.GN_ERR_VARIANT), (dict(q=A + 8), gs.GN_ERR_ALIGN), (dict(lse=E + 2), gs.GN_ERR_ALIGN),
    (dict(k_token=132), gs.GN_ERR_ALIGN), (dict(cu_k=F + 1), gs.GN_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,code", BAD + [(dict(out=A + 256), gs.GN_ERR_ALIAS), (dict(lse=B), gs.GN_ERR_ALIAS),
                                           (dict(lse=D), gs.GN_ERR_ALIAS)])
def test_attention_refuses(kw, code):
    assert attn(**kw) == code


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(dout=None), gs.GN_ERR_NULL), (dict(dk=None), gs.GN_ERR_NULL), (dict(ws=None), gs.GN_ERR_NULL),
    (dict(dout=G + 2), gs.GN_ERR_ALIGN), (dict(dt=12), gs.GN_ERR_ALIGN), (dict(ws=H + 256 * S + 16), gs.GN_ERR_ALIGN),
    (dict(dt=0), gs.GN_ERR_SHAPE), (dict(dq=A), gs.GN_ERR_ALIAS), (dict(dv=H + 64 * S), gs.GN_ERR_ALIAS),
    (dict(dk=D), gs.GN_ERR_ALIAS), (dict(ws=G), gs.GN_ERR_ALIAS), (dict(wsb=64), gs.GN_ERR_WORKSPACE)])
def test_attention_backward_refuses(kw, code):
    assert attn(backward=True, **kw) == code


def test_workspace_sizes():
    assert block.gn_attn_packed_workspace_bytes(100, 4) >= 1600
    assert block.gn_attn_packed_workspace_bytes(-1, 4) == 0
    assert block.gn_attn_packed_workspace_bytes(10, 0) == 0
    assert gs.lib().gn_layer_norm_workspace_bytes(-1, 64) == 0
    assert gs.lib().gn_layer_norm_workspace_bytes(8, 0) == 0


def test_tensors_off_the_gpu_give_none():
    x = torch.zeros(4, 64)
    assert block.layer_norm(x) is None
    assert block.layer_norm_backward(x, x, x[:, 0], x[:, 0]) is None
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    assert block.rope_nd(q, q, torch.zeros(4, 1), [64]) is None
    assert block.attention_packed(q, q, q) is None
    assert block.attention_packed_backward(q, q, q, q, q, torch.zeros(2, 4)) is None


def test_reference_gradients_against_differences():
    """The formulas' gradients, which the GPU tests hold the kernels to,
    against central differences of the formulas' outputs."""
    gen = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    step = 1e-5

    def differences(f, t):
        g = torch.zeros_like(t)
        for n in range(t.numel()):
            keep = t.view(-1)[n].item()
            t.view(-1)[n] = keep + step
            up = f()
            t.view(-1)[n] = keep - step
            g.view(-1)[n] = (up - f()) / (2 * step)
            t.view(-1)[n] = keep
        return g

    x, w, b, dy = rand(3, 10), rand(10), rand(10), rand(3, 10)
    r = br.layer_norm(x, w, b, 1e-3, dy)
    for t, name in ((x, "dx"), (w, "dw"), (b, "db")):
        d = differences(lambda: float((br.layer_norm(x, w, b, 1e-3)["y"][0] * dy).sum()), t)
        assert (d - r[name][0]).abs().max() < 1e-7, name

    q, k, v, do = rand(7, 4, 8), rand(9, 2, 8), rand(9, 2, 8), rand(7, 4, 8)
    how = dict(cu_q=[0, 3, 7], cu_k=[0, 2, 9], causal=True, prefix=[0, 4], slopes=torch.tensor([0.1, 0.2, 0.3, 0.4]),
               cap=2.0)
    r = br.attention(q, k, v, **how, dout=do)
    for t, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        d = differences(lambda: float((br.attention(q, k, v, **how)["out"][0] * do).sum()), t)
        assert (d - r[name][0]).abs().max() < 1e-7, name

    pos = rand(5, 2) * 10
    a, g = rand(5, 2, 12), rand(5, 2, 12)
    for inter in (True, False):
        d = differences(lambda: float((br.rope(a, pos, [4, 6], 100.0, inter, False)[0] * g).sum()), a)
        assert (d - br.rope(g, pos, [4, 6], 100.0, inter, True)[0]).abs().max() < 1e-7
