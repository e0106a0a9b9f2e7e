"""RMS norm and the paged cache on the host, without a GPU: every kind of unsupported
input is refused with its status before any CUDA call, and the 64-bit references that
the GPU tests use are checked against differences and against plain loops."""
import ctypes
import math

import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from channels_last_groupnorm_gb300 import serve
from tests import serve_ref as sr

# stand-in device addresses, far apart (never dereferenced: every call below is refused first)
A, B, C, D, E, F, G, H, I, J, K, M = (0x1000000000 * n for n in range(1, 13))
S = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    gnbuild.build()


def strides(*values):
    return (ctypes.c_int64 * 8)(*values)


def norm(**kw):
    a = dict(x=A, r=B, w=C, y=D, t=E, s=None, rstd=F, rows=16, cols=64, xs=64, rs=64, ys=64, ts=64, eps=1e-6, fmt=0, wfmt=2)
    a.update(kw)
    st = None if a.get("none") else strides(0, a["xs"], a.get("ro", 0), a["rs"], a.get("yo", 0), a["ys"], 0, a["ts"])
    return gs.lib().gn_rms_norm(a["x"], a["r"], a["w"], a["y"], a["t"], a["s"], a["rstd"], a["rows"], a["cols"],
                                a.get("inner", 1 << 40), st, a["eps"], a["fmt"], a["wfmt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), gs.GN_ERR_NULL), (dict(y=None), gs.GN_ERR_NULL), (dict(r=None), gs.GN_ERR_NULL), (dict(t=None), gs.GN_ERR_NULL),
    (dict(none=True), gs.GN_ERR_NULL), (dict(fmt=3), gs.GN_ERR_FORMAT), (dict(wfmt=-1), gs.GN_ERR_FORMAT),
    (dict(rows=-1), gs.GN_ERR_SHAPE), (dict(cols=0), gs.GN_ERR_CHANNELS), (dict(cols=16385, xs=S, rs=S, ys=S, ts=S), gs.GN_ERR_CHANNELS),
    (dict(xs=63), gs.GN_ERR_SHAPE), (dict(ys=0), gs.GN_ERR_SHAPE), (dict(ts=32), gs.GN_ERR_SHAPE), (dict(rows=1 << 60), gs.GN_ERR_SHAPE),
    (dict(inner=0), gs.GN_ERR_SHAPE), (dict(eps=math.nan), gs.GN_ERR_EPS), (dict(eps=-1.0), gs.GN_ERR_EPS),
    (dict(x=A + 1), gs.GN_ERR_ALIGN), (dict(s=G + 2), gs.GN_ERR_ALIGN), (dict(w=C + 2), gs.GN_ERR_ALIGN), (dict(rstd=F + 1), gs.GN_ERR_ALIGN),
    (dict(y=A), gs.GN_ERR_ALIAS), (dict(y=B + 128), gs.GN_ERR_ALIAS), (dict(t=A + 128), gs.GN_ERR_ALIAS), (dict(t=B, ts=128), gs.GN_ERR_ALIAS),
    (dict(y=E), gs.GN_ERR_ALIAS), (dict(s=F), gs.GN_ERR_ALIAS), (dict(s=A + 64), gs.GN_ERR_ALIAS), (dict(rstd=D), gs.GN_ERR_ALIAS),
    (dict(w=D), gs.GN_ERR_ALIAS), (dict(w=E), gs.GN_ERR_ALIAS), (dict(x=A, y=A, s=G, r=None, t=None), gs.GN_ERR_ALIAS),
])
def test_rms_norm_refuses(kw, code):
    assert norm(**kw) == code


def norm_grad(**kw):
    a = dict(dy=A, t=B, w=C, rstd=D, dt=E, dx=F, dw=G, ws=H, wsb=1 << 30, rows=16, cols=64, gs=64, ts=64, bs=64, xs=64, fmt=0, wfmt=2)
    a.update(kw)
    return gs.lib().gn_rms_norm_backward(a["dy"], a["t"], a["w"], a["rstd"], a["dt"], a["dx"], a["dw"], a["rows"], a["cols"],
                                         a.get("inner", 1 << 40), strides(0, a["gs"], 0, a["ts"], 0, a["bs"], 0, a["xs"]),
                                         a["fmt"], a["wfmt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), gs.GN_ERR_NULL), (dict(t=None), gs.GN_ERR_NULL), (dict(rstd=None), gs.GN_ERR_NULL), (dict(dx=None), gs.GN_ERR_NULL),
    (dict(dw=None), gs.GN_ERR_NULL), (dict(w=None), gs.GN_ERR_NULL), (dict(ws=None), gs.GN_ERR_NULL), (dict(fmt=4), gs.GN_ERR_FORMAT),
    (dict(rows=-2), gs.GN_ERR_SHAPE), (dict(cols=0), gs.GN_ERR_CHANNELS), (dict(gs=3), gs.GN_ERR_SHAPE), (dict(xs=0), gs.GN_ERR_SHAPE),
    (dict(ws=H + 8), gs.GN_ERR_ALIGN), (dict(dt=E + 1), gs.GN_ERR_ALIGN), (dict(dx=A + 2), gs.GN_ERR_ALIAS), (dict(dx=E, xs=128), gs.GN_ERR_ALIAS),
    (dict(dx=D), gs.GN_ERR_ALIAS), (dict(dw=F), gs.GN_ERR_ALIAS), (dict(ws=A), gs.GN_ERR_ALIAS), (dict(dw=H), gs.GN_ERR_ALIAS),
])
def test_rms_norm_backward_refuses(kw, code):
    assert norm_grad(**kw) == code


# gn_cache: 7 pages of 16 tokens, 2 heads, 32 channels, heads first
def cache(**kw):
    a = dict(kp=A, vp=B, ks=C, vs=D, k=(1024, 32, 512), v=(1024, 32, 512), table=E, lengths=F, cu=G, pages=7, width=3, seqs=2,
             size=16, heads=2, dim=32)
    a.update(kw)
    return serve._CACHE.pack(a["kp"] or 0, a["vp"] or 0, a["ks"] or 0, a["vs"] or 0, *a["k"], *a["v"], a["table"] or 0,
                             a["lengths"] or 0, a["cu"] or 0, a["pages"], a["width"], a["seqs"], a["size"], a["heads"], a["dim"])


BAD_CACHES = [
    (dict(kp=None), gs.GN_ERR_NULL), (dict(vp=None), gs.GN_ERR_NULL), (dict(ks=None), gs.GN_ERR_NULL), (dict(vs=None), gs.GN_ERR_NULL),
    (dict(table=None), gs.GN_ERR_NULL), (dict(lengths=None), gs.GN_ERR_NULL), (dict(seqs=0), gs.GN_ERR_SHAPE),
    (dict(seqs=(1 << 20) + 1), gs.GN_ERR_SHAPE), (dict(pages=0), gs.GN_ERR_SHAPE), (dict(pages=1 << 31), gs.GN_ERR_SHAPE),
    (dict(width=0), gs.GN_ERR_SHAPE), (dict(width=1 << 27), gs.GN_ERR_SHAPE), (dict(size=12), gs.GN_ERR_CHANNELS),
    (dict(size=0), gs.GN_ERR_CHANNELS), (dict(size=264), gs.GN_ERR_CHANNELS), (dict(heads=0), gs.GN_ERR_CHANNELS),
    (dict(dim=24), gs.GN_ERR_CHANNELS), (dict(dim=144), gs.GN_ERR_CHANNELS), (dict(dim=0), gs.GN_ERR_CHANNELS),
    (dict(kp=A + 8), gs.GN_ERR_ALIGN), (dict(v=(1024, 40, 512)), gs.GN_ERR_ALIGN), (dict(cu=G + 2), gs.GN_ERR_ALIGN),
    (dict(vs=D + 1), gs.GN_ERR_ALIGN), (dict(k=(1024, 16, 512)), gs.GN_ERR_SHAPE), (dict(k=(1008, 32, 512)), gs.GN_ERR_SHAPE),
    (dict(v=(0, 32, 512)), gs.GN_ERR_SHAPE), (dict(v=(-1024, 32, 512)), gs.GN_ERR_SHAPE), (dict(k=(1 << 62, 32, 512)), gs.GN_ERR_SHAPE),
    (dict(k=(32, 224, 48)), gs.GN_ERR_SHAPE),
]


def append(cache_bytes=None, null=False, **kw):
    a = dict(q=H, k=I, v=J, out=K, q_s=(128, 32), k_s=(64, 32), v_s=(64, 32), o_s=(128, 32), tokens=6, pos=M, axes=[8, 24], theta=1e4,
             heads=4, pfmt=0, fmt=0)
    a.update(kw)
    axes = (ctypes.c_int64 * 9)(*a["axes"])
    args = serve._APPEND.pack(a["q"] or 0, a["k"] or 0, a["v"] or 0, a["out"] or 0, *a["q_s"], *a["k_s"], *a["v_s"], *a["o_s"], a["tokens"],
                              a["pos"] or 0, 0 if a.get("no_axes") else ctypes.addressof(axes), a["theta"], a["heads"], len(a["axes"]),
                              a["pfmt"], 1, a["fmt"])
    return gs.lib().gn_cache_append(None if null else (cache_bytes or cache()), args, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_append_and_attention_refuse_caches(kw, code):
    assert append(cache(**kw)) == code
    assert attend(cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(null=True), gs.GN_ERR_NULL), (dict(k=None), gs.GN_ERR_NULL), (dict(v=None), gs.GN_ERR_NULL), (dict(q=None), gs.GN_ERR_NULL),
    (dict(out=None), gs.GN_ERR_NULL), (dict(pos=None), gs.GN_ERR_NULL), (dict(no_axes=True), gs.GN_ERR_NULL),
    (dict(tokens=-1), gs.GN_ERR_SHAPE), (dict(tokens=(1 << 30) + 2), gs.GN_ERR_SHAPE), (dict(fmt=3), gs.GN_ERR_FORMAT),
    (dict(pfmt=3), gs.GN_ERR_FORMAT), (dict(heads=-1), gs.GN_ERR_CHANNELS), (dict(heads=65537), gs.GN_ERR_CHANNELS),
    (dict(axes=[2] * 9), gs.GN_ERR_CHANNELS), (dict(axes=[7]), gs.GN_ERR_CHANNELS), (dict(axes=[34]), gs.GN_ERR_CHANNELS),
    (dict(axes=[20, 20]), gs.GN_ERR_CHANNELS), (dict(theta=0.0), gs.GN_ERR_EPS), (dict(theta=math.inf), gs.GN_ERR_EPS),
    (dict(theta=math.nan), gs.GN_ERR_EPS), (dict(k=I + 1), gs.GN_ERR_ALIGN), (dict(pos=M + 2), gs.GN_ERR_ALIGN),
    (dict(o_s=(128, 31)), gs.GN_ERR_SHAPE), (dict(o_s=(64, 32)), gs.GN_ERR_SHAPE), (dict(k_s=(-64, 32)), gs.GN_ERR_SHAPE),
    (dict(out=H + 64), gs.GN_ERR_ALIAS), (dict(out=H, o_s=(256, 32)), gs.GN_ERR_ALIAS), (dict(out=I), gs.GN_ERR_ALIAS),
    (dict(out=M), gs.GN_ERR_ALIAS), (dict(k=A), gs.GN_ERR_ALIAS), (dict(v=C), gs.GN_ERR_ALIAS), (dict(out=F), gs.GN_ERR_ALIAS),
    (dict(cache_bytes=dict(vp=A)), gs.GN_ERR_ALIAS), (dict(cache_bytes=dict(vp=A + 512)), gs.GN_ERR_ALIAS),
    (dict(cache_bytes=dict(vs=C + 8)), gs.GN_ERR_ALIAS), (dict(cache_bytes=dict(ks=B)), gs.GN_ERR_ALIAS),
    (dict(cache_bytes=dict(table=A + 16)), gs.GN_ERR_ALIAS), (dict(cache_bytes=dict(lengths=D)), gs.GN_ERR_ALIAS),
    # slices of one buffer whose last page runs into the next one's first
    (dict(cache_bytes=dict(vp=A + 1024, k=(2032, 32, 512), v=(2032, 32, 512))), gs.GN_ERR_ALIAS),
    (dict(cache_bytes=dict(vp=A + 64, k=(2032, 128, 32), v=(2032, 128, 32))), gs.GN_ERR_ALIAS),
    (dict(cache_bytes=dict(cu=None, seqs=4)), gs.GN_ERR_SHAPE),
])
def test_append_refuses(kw, code):
    kw = dict(kw)
    if "cache_bytes" in kw:
        kw["cache_bytes"] = cache(**kw["cache_bytes"])
    assert append(**kw) == code


def attend(cache_bytes=None, null=False, **kw):
    a = dict(q=H, out=I, lse=J, slopes=K, q_s=(128, 32), tokens=6, scale=0.2, cap=0.0, heads=4, causal=1, fmt=0, ws=M, wsb=1 << 30)
    a.update(kw)
    args = serve._ATTN.pack(a["q"] or 0, a["out"] or 0, a["lse"] or 0, a["slopes"] or 0, *a["q_s"], a["tokens"], a["scale"], a["cap"],
                            a["heads"], a["causal"], a["fmt"])
    return gs.lib().gn_attn_cached(None if null else (cache_bytes or cache()), args, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(null=True), gs.GN_ERR_NULL), (dict(q=None), gs.GN_ERR_NULL), (dict(out=None), gs.GN_ERR_NULL), (dict(lse=None), gs.GN_ERR_NULL),
    (dict(ws=None), gs.GN_ERR_NULL), (dict(tokens=-1), gs.GN_ERR_SHAPE), (dict(fmt=2), gs.GN_ERR_FORMAT), (dict(heads=3), gs.GN_ERR_CHANNELS),
    (dict(heads=0), gs.GN_ERR_CHANNELS), (dict(heads=1026), gs.GN_ERR_CHANNELS), (dict(scale=math.nan), gs.GN_ERR_EPS),
    (dict(cap=-1.0), gs.GN_ERR_EPS), (dict(cap=math.inf), gs.GN_ERR_EPS), (dict(q=H + 8), gs.GN_ERR_ALIGN), (dict(q_s=(132, 32)), gs.GN_ERR_ALIGN),
    (dict(ws=M + 16), gs.GN_ERR_ALIGN), (dict(lse=J + 2), gs.GN_ERR_ALIGN), (dict(q_s=(128, 16)), gs.GN_ERR_SHAPE),
    (dict(out=H), gs.GN_ERR_ALIAS), (dict(lse=I), gs.GN_ERR_ALIAS), (dict(ws=A), gs.GN_ERR_ALIAS), (dict(out=E), gs.GN_ERR_ALIAS),
    (dict(ws=I), gs.GN_ERR_ALIAS), (dict(lse=K), gs.GN_ERR_ALIAS),
])
def test_attention_refuses(kw, code):
    assert attend(**kw) == code


def test_tensors_off_the_gpu_give_none():
    x = torch.zeros(4, 64)
    assert gn.rms_norm(x) is None and gn.rms_norm_backward(x, x, x[:, 0]) is None
    pages = torch.zeros(3, 16, 2, 32, dtype=torch.uint8).view(sr.E4M3)
    scales, table, lengths = torch.ones(3, 2), torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 32, dtype=torch.bfloat16)
    assert gn.cache_append(k, k, pages, pages, scales, scales, table, lengths) is None
    assert gn.attention_cached(k, pages, pages, scales, scales, table, lengths) is None


def test_workspace_of_unsupported_shapes():
    assert gn.gn_rms_norm_workspace_bytes(-1, 64) == 0 and gn.gn_rms_norm_workspace_bytes(4, 0) == 0
    for a in ((-1, 1, 4, 2, 64), (4, 0, 4, 2, 64), (4, 1, 4, 3, 64), (4, 1, 4, 2, 24), (4, 1, 2000, 2, 64)):
        assert gn.gn_attn_cached_workspace_bytes(*a) == 0


def test_reference_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, dy, dt = rand(3, 10), rand(10), rand(3, 10), rand(3, 10)
    r = sr.rms_norm(x, w, 1e-3, dy=dy, dtotal=dt)
    loss = lambda: float((sr.rms_norm(x, w, 1e-3)["y"][0] * dy).sum() + (x * dt).sum())  # noqa: E731
    for t, name in ((x, "dx"), (w, "dw")):
        for n in range(t.numel()):
            keep = t.view(-1)[n].item()
            t.view(-1)[n] = keep + 1e-5
            up = loss()
            t.view(-1)[n] = keep - 1e-5
            d = (up - loss()) / 2e-5
            t.view(-1)[n] = keep
            assert abs(d - float(r[name][0].view(-1)[n])) < 1e-7, name


def test_reference_cast_and_scales():
    x = torch.cat([torch.randn(5000, generator=torch.Generator().manual_seed(1)).double() * 10,
                   torch.arange(-480, 481).double() / 512, torch.tensor([0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    assert torch.equal(sr.cast_e4m3(x), x.float().to(sr.E4M3).double())
    assert sr.least_scale(448.0) == 1.0 and sr.least_scale(448.0001) == 2.0 and sr.least_scale(3.5) == 2.0 ** -7
    assert sr.least_scale(0.0) == sr.least_scale(1e-38) == 2.0 ** -100 and math.isnan(sr.least_scale(math.inf))


def test_reference_attention_against_loops():
    cache = sr.Cache([5, 40], 16, 1, 16, seed=1, device="cpu")
    q = torch.randn(4, 2, 16, generator=torch.Generator().manual_seed(2)).bfloat16()
    got = sr.attention(q, cache, [0, 1, 4])["out"][0]
    for t, (s, last) in enumerate([(0, 4), (1, 37), (1, 38), (1, 39)]):
        k, v = cache.values("k", s)[:last + 1, 0], cache.values("v", s)[:last + 1, 0]
        for h in range(2):
            p = torch.softmax(k @ q[t, h].double() / 4.0, 0)
            assert torch.allclose(got[t, h], p @ v, rtol=1e-12, atol=1e-12)
