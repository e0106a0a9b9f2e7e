"""The transformer-block operators on the GPU against their definitions in 64
bits (tests/block_ref.py, which also derives how far each output may be)."""
import math

import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from tests import block_ref as br
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    gs.lib()
    yield
    gu.assert_clean_device()


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale + shift).to(dtype).cuda()


def guarded(shape, dtype):
    """A contiguous tensor inside a buffer of a known value, and a check that
    nothing around it was written."""
    n = math.prod(shape)
    buf = torch.full((n + 512,), -7.0, dtype=dtype, device="cuda")

    def clean():
        assert bool((buf[:256] == -7.0).all() and (buf[256 + n:] == -7.0).all())
    return buf[256:256 + n].view(shape), clean


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 6144), (5, 8), (257, 128), (1000, 64), (33, 40), (129, 1003),
                                       (2, 16384), (3, 16383), (700, 1536), (19, 5000), (311, 12288), (4099, 16)])
@pytest.mark.parametrize("weight", [None, "own", F32])
def test_layer_norm(rows, cols, dtype, weight):
    x = rand((rows, cols), dtype, rows + cols, 2.0, 1.5)
    wt = dtype if weight == "own" else weight
    w = b = None
    if wt is not None:
        w, b = rand((cols,), wt, 1, 0.3, 1.0), rand((cols,), wt, 2, 0.5)
    dy = rand((rows, cols), dtype, 3)
    out, clean = guarded((rows, cols), dtype)
    y, mean, rstd = gn.layer_norm(x, w, b, eps=1e-3, out=out)
    grad, clean_grad = guarded((rows, cols), dtype)
    dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w, out=grad)
    torch.cuda.synchronize()
    assert y is out and dx is grad
    clean()
    clean_grad()
    want = br.layer_norm(x, w, b, 1e-3, dy)
    got = dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
    for name, (value, bound) in want.items():
        br.check(got[name], value, bound, f"{name} {rows}x{cols}")
    if w is None:
        assert dw is None and db is None


@pytest.mark.parametrize("rows,cols,wide,dtype", [
    (40001, 128, 128, FP), (130000, 32, 32, F32), (2000, 6144, 6144, BF), (1301, 8192, 8192, BF), (700, 12288, 12288, BF),
    (1999, 1000, 1024, BF), (5003, 520, 520, FP), (9000, 264, 272, F32), (64000, 64, 72, BF)])
def test_layer_norm_many_rows(rows, cols, wide, dtype):
    """Enough rows for the streamed kernels, rows end to end and out of a wider tensor."""
    x = rand((rows, wide), dtype, 1, 2.0, 1.0)[:, :cols]
    dy = rand((rows, wide), dtype, 2)[:, :cols]
    for w, b in ((rand((cols,), F32, 3, 0.3, 1.0), rand((cols,), F32, 4)), (None, None)):
        y, mean, rstd = gn.layer_norm(x, w, b)
        dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
        got = dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
        for name, (value, bound) in br.layer_norm(x, w, b, 1e-6, dy).items():
            br.check(got[name], value, bound, name)
        again = gn.layer_norm_backward(dy, x, mean, rstd, w)
        assert all(p is q or torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("rows,cols,wide,dtype", [
    (613, 6152, 6152, BF), (1217, 6400, 6416, FP), (1500, 12288, 12296, BF), (608, 9000, 9000, FP), (700, 6144, 6144, F32),
    (1999, 3080, 3092, F32)])
def test_layer_norm_wide_rows_backward(rows, cols, wide, dtype):
    """Rows of which the backward pass holds four slots a thread: one batch short of and past the ring's turns."""
    x = rand((rows, wide), dtype, 5, 2.0, 1.0)[:, :cols]
    dy = rand((rows, wide), dtype, 6)[:, :cols]
    for w, b in ((rand((cols,), F32, 7, 0.3, 1.0), rand((cols,), F32, 8)), (None, None)):
        y, mean, rstd = gn.layer_norm(x, w, b)
        dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
        got = dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
        for name, (value, bound) in br.layer_norm(x, w, b, 1e-6, dy).items():
            br.check(got[name], value, bound, name)
        # in place over dy, and the same bits again
        onto = dy.clone()
        again = gn.layer_norm_backward(onto, x, mean, rstd, w, out=onto)
        assert all(p is q or torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("rows,cols,wide,start,dtype", [
    (300000, 1, 1, 0, BF), (300000, 5, 5, 3, FP), (240000, 7, 9, 1, F32), (60001, 67, 67, 0, BF), (40000, 131, 131, 1, FP),
    (30011, 131, 140, 5, BF), (9001, 257, 257, 0, F32), (9000, 514, 515, 1, FP), (5003, 1001, 1001, 7, BF), (5000, 1003, 1003, 0, F32),
    (2500, 2050, 2050, 0, BF), (1301, 6143, 6143, 1, FP), (1300, 6150, 6157, 2, BF), (700, 10007, 10007, 0, FP),
    (700, 12001, 12001, 3, BF), (640, 5001, 5003, 1, F32), (640, 15001, 15001, 0, FP), (40000, 128, 128, 1, BF),
    (2003, 200, 203, 1, F32), (3001, 131, 131, 0, FP), (40001, 133, 133, 0, F32), (9999, 515, 515, 2, F32), (2000, 2051, 2051, 0, F32),
    (5001, 1003, 1010, 3, BF), (700, 12002, 12002, 0, F32)])
def test_layer_norm_many_rows_that_begin_anywhere(rows, cols, wide, start, dtype):
    """Many rows that are not whole vectors, or lie at any element, end to end and out of a wider tensor."""
    def lie(seed, scale, shift=0.0):
        return rand((rows * wide + start,), dtype, seed, scale, shift)[start:].view(rows, wide)[:, :cols]
    x, dy = lie(5, 2.0, 1.0), lie(6, 1.0)
    for w, b in ((rand((cols,), F32, 7, 0.3, 1.0), rand((cols,), F32, 8)), (rand((cols,), dtype, 7, 0.3, 1.0), None), (None, None)):
        out, clean = guarded((rows, cols), dtype)
        y, mean, rstd = gn.layer_norm(x, w, b, out=out)
        grad, clean_grad = guarded((rows, cols), dtype)
        dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w, out=grad)
        clean()
        clean_grad()
        got = dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
        for name, (value, bound) in br.layer_norm(x, w, b, 1e-6, dy).items():
            br.check(got[name], value, bound, name)
    # in place on rows of a wider tensor, whose other elements stay; the same bits
    whole = torch.full((rows * (wide + 2) + start,), -7.0, dtype=dtype, device="cuda")
    onto = whole[start:].view(rows, wide + 2)[:, 1:1 + cols]
    onto.copy_(dy)
    keep = whole.clone()
    again = gn.layer_norm_backward(onto, x, mean, rstd, w, out=onto)
    assert torch.equal(again[0], dx)
    onto.copy_(keep[start:].view(rows, wide + 2)[:, 1:1 + cols])
    assert torch.equal(whole, keep)


@pytest.mark.parametrize("cols,start,wide", [(64, 0, 64 + 8), (64, 3, 80), (129, 1, 200), (512, 8, 1024)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_norm_of_column_slices(cols, start, wide, dtype):
    x = rand((37, wide), dtype, 5)[:, start:start + cols]
    dy = rand((37, wide + 1), dtype, 6)[:, :cols]
    w, b = rand((cols,), F32, 7, 0.2, 1.0), rand((cols,), F32, 8)
    y, mean, rstd = gn.layer_norm(x, w, b)
    dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
    want = br.layer_norm(x, w, b, 1e-6, dy)
    for name, got in dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db).items():
        br.check(got, *want[name], name)


@pytest.mark.parametrize("tokens,heads,cols,dtype", [(3, 5, 64, BF), (700, 24, 128, FP), (9, 1, 40, F32), (4000, 8, 72, BF),
                                                     (1, 7, 33, F32)])
def test_layer_norm_of_some_heads_of_a_projection(tokens, heads, cols, dtype):
    """Rows with two strides: [tokens, heads, cols] slices of a wider tensor."""
    qkv, grads = rand((tokens, heads + 3, cols), dtype, 1, 2.0, 1.0), rand((tokens, heads + 1, cols), dtype, 2)
    x, dy = qkv[:, 2:2 + heads], grads[:, :heads]
    w, b = rand((cols,), F32, 3, 0.2, 1.0), rand((cols,), F32, 4)
    y, mean, rstd = gn.layer_norm(x, w, b)
    dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
    assert y.is_contiguous() and mean.shape == (tokens, heads)
    want = br.layer_norm(x.reshape(-1, cols), w, b, 1e-6, dy.reshape(-1, cols))
    got = dict(y=y.view(-1, cols), mean=mean.view(-1), rstd=rstd.view(-1), dx=dx.view(-1, cols), dw=dw, db=db)
    for name, (value, bound) in want.items():
        br.check(got[name], value, bound, name)
    # in place, and onto slices of another tensor
    keep = qkv.clone()
    assert gn.layer_norm(x, w, b, out=x)[0] is x
    assert torch.equal(x, y) and torch.equal(qkv[:, :2], keep[:, :2]) and torch.equal(qkv[:, 2 + heads:], keep[:, 2 + heads:])
    onto = torch.zeros((tokens, heads + 1, cols), dtype=dtype, device="cuda")
    gn.layer_norm_backward(dy, keep[:, 2:2 + heads], mean, rstd, w, out=onto[:, 1:])
    assert torch.equal(onto[:, 1:], dx) and not onto[:, 0].any()


def test_layer_norm_shapes_in_place_and_repeated():
    x = rand((3, 5, 7, 256), BF, 9, 2.0, 3.0)
    w, b = rand((256,), BF, 10), rand((256,), BF, 11)
    y, mean, rstd = gn.layer_norm(x, w, b)
    assert y.shape == x.shape and mean.shape == x.shape[:-1]
    again = x.clone()
    assert gn.layer_norm(again, w, b, out=again)[0] is again
    assert torch.equal(again, y)
    no_bias = gn.layer_norm(x, w)[0]
    br.check(no_bias.view(-1, 256), *br.layer_norm(x.view(-1, 256), w, None, 1e-6)["y"], "weight alone")
    dy = rand(x.shape, BF, 12)
    first = gn.layer_norm_backward(dy, x, mean, rstd, w)
    second = gn.layer_norm_backward(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    onto = dy.clone()
    third = gn.layer_norm_backward(onto, x, mean, rstd, w, out=onto)
    assert all(torch.equal(p, q) for p, q in zip(first, third))


def test_layer_norm_edges():
    y, mean, rstd = gn.layer_norm(torch.empty(0, 64, device="cuda", dtype=BF))
    assert y.shape == (0, 64) and mean.shape == (0,)
    w = torch.ones(64, device="cuda")
    dx, dw, db = gn.layer_norm_backward(y, y, mean, rstd, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    # a constant row: no spread, eps alone; a row with a NaN keeps it to itself
    x = torch.full((3, 100), 5.0, device="cuda")
    x[1, 3] = math.nan
    y, mean, rstd = gn.layer_norm(x, eps=1e-6)
    assert not y[0].any() and torch.isnan(y[1]).all() and not y[2].any()
    assert torch.allclose(rstd[0], torch.tensor(1e3, device="cuda"), rtol=1e-6)
    # far from zero: the variance is taken about the mean
    x = rand((64, 1000), F32, 13, 1.0, 4096.0)
    for name, got in zip(("y", "mean", "rstd"), gn.layer_norm(x)):
        br.check(got, *br.layer_norm(x, None, None, 1e-6)[name], name)


def test_layer_norm_not_supported():
    x = rand((4, 64), BF, 1)
    w = torch.ones(64, device="cuda")
    assert gn.layer_norm(x.double()) is None
    assert gn.layer_norm(x, bias=w) is None
    assert gn.layer_norm(x, w, w.to(BF)) is None
    assert gn.layer_norm(x, w[:32]) is None
    assert gn.layer_norm(x.t()) is None
    assert gn.layer_norm(x.clone().requires_grad_()) is None
    assert gn.layer_norm(x, out=x[:2]) is None
    with pytest.warns(UserWarning):
        assert gn.layer_norm(torch.zeros(1, 16385, device="cuda")) is None
    with torch.no_grad():
        assert gn.layer_norm(x.clone().requires_grad_()) is not None
    m = torch.zeros(4, device="cuda")
    assert gn.layer_norm_backward(x, x, m.to(BF), m) is None
    assert gn.layer_norm_backward(x[:3], x, m, m) is None


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def places(tokens, axes, kind, far=0):
    t = torch.arange(tokens)[:, None] * torch.tensor([1, 3, 7, 2, 5, 4, 9, 8])[None, :axes] + far
    if kind == "fp32":
        return (t * 0.64 + 0.125).float().cuda()
    return t.to(getattr(torch, kind)).cuda()


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("tokens,h,hk,dim,axes,inter,kind", [
    (1, 48, 8, 128, [32, 32, 32, 32], True, "int32"), (5, 3, 1, 128, [16, 56, 56], False, "fp32"),
    (300, 2, 2, 64, [64], True, "int64"), (77, 4, 2, 72, [20, 22, 22], False, "int32"),
    (33, 1, 1, 30, [2, 4, 6], True, "int32"), (9, 5, 5, 31, [10, 10], False, "fp32"),
    (2, 7, 1, 256, [128, 128], True, "int64"), (1025, 6, 3, 136, [24, 36, 36], True, "fp32"),
    (64, 2, 1, 96, [12, 12, 12, 12, 12, 12, 12, 12], False, "int32")])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(tokens, h, hk, dim, axes, inter, kind, inverse, dtype):
    q, k = rand((tokens, h, dim), dtype, 1), rand((tokens, hk, dim), dtype, 2)
    pos = places(tokens, len(axes), kind)
    (qo, c0), (ko, c1) = guarded(q.shape, dtype), guarded(k.shape, dtype)
    got = gn.rope_nd(q, k, pos, axes, theta=2000.0, interleaved=inter, inverse=inverse, out=(qo, ko))
    torch.cuda.synchronize()
    assert got[0] is qo and got[1] is ko
    c0()
    c1()
    for x, y in ((q, qo), (k, ko)):
        br.check(y, *br.rope(x, pos, axes, 2000.0, inter, inverse), "rope")
    rest = sum(axes)
    assert torch.equal(qo[..., rest:], q[..., rest:])


@pytest.mark.parametrize("inter", [False, True])
def test_rope_far_positions(inter):
    q = rand((200, 2, 64), F32, 3)
    for kind, far in (("int32", 1 << 30), ("int64", 1 << 36), ("fp32", 1 << 20)):
        pos = places(200, 2, kind, far)
        got, none = gn.rope_nd(q, None, pos, [32, 32], theta=1e6, interleaved=inter)
        assert none is None
        want, bound = br.rope(q, pos, [32, 32], 1e6, inter, False)
        # position x rate in fp64 on both sides: 2^-52 of the angle
        br.check(got, want, bound + far * 2.0 ** -51 * q.abs().amax(), kind)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_in_place_on_slices_of_a_projection(dtype):
    qkv = rand((50, 4 + 2 + 2, 128), dtype, 4)
    keep = qkv.clone()
    pos = places(50, 3, "int32")
    q, k = qkv[:, :4], qkv[:, 4:6]
    want = gn.rope_nd(keep[:, :4], keep[:, 4:6], pos, [16, 56, 56])
    got = gn.rope_nd(q, k, pos, [16, 56, 56], out=(q, k))
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 6:], keep[:, 6:])
    back = gn.rope_nd(want[0], want[1], pos, [16, 56, 56], inverse=True)
    size = 4 * br.half_step(dtype) + 48 * br.U32             # two roundings of values up to |a| + |b|
    assert float((back[0].float() - keep[:, :4].float()).abs().max()) <= size * 2 * float(keep.abs().max())
    # heads before tokens, and channels that do not start on a 16-byte boundary
    odd = rand((2, 50, 133), dtype, 5).transpose(0, 1)[..., 1:129]
    got, _ = gn.rope_nd(odd, None, pos, [16, 56, 56], interleaved=False)
    br.check(got, *br.rope(odd, pos, [16, 56, 56], 1e4, False, False), "strided")


def test_rope_not_supported():
    q, pos = rand((4, 2, 64), BF, 1), places(4, 1, "int32")
    assert gn.rope_nd(q, None, pos, [64])[0] is not None
    assert gn.rope_nd(q, None, pos.double(), [64]) is None
    assert gn.rope_nd(q, None, pos[:3], [64]) is None
    assert gn.rope_nd(q, q.float(), pos, [64]) is None
    assert gn.rope_nd(q, None, pos, [32, 32]) is None
    assert gn.rope_nd(q.clone().requires_grad_(), None, pos, [64]) is None
    with pytest.warns(UserWarning):
        assert gn.rope_nd(q, None, pos, [66]) is None
    empty = gn.rope_nd(q[:0], None, pos[:0], [64])
    assert empty[0].shape == (0, 2, 64)


# ---------------------------------------------------------------------------
# attention of packed documents
# ---------------------------------------------------------------------------
def ends(lens, start=0):
    e = [start]
    for n in lens:
        e.append(e[-1] + n)
    return e


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(q, k, v, cu_q, cu_k, dout=None, prefix=None, **how):
    """The package's outputs by name, for lists of ends."""
    how = dict(how, prefix=None if prefix is None else i32(prefix))
    r = gn.attention_packed(q, k, v, i32(cu_q), i32(cu_k), **how)
    assert r is not None, "refused a supported input"
    got = dict(out=r[0], lse=r[1])
    if dout is not None:
        g = gn.attention_packed_backward(dout, q, k, v, r[0], r[1], i32(cu_q), i32(cu_k), **how)
        assert g is not None, "refused a supported input"
        got |= dict(dq=g[0], dk=g[1], dv=g[2])
    torch.cuda.synchronize()
    gu.assert_clean_device()
    return got


def against_reference(got, q, k, v, cu_q, cu_k, dout=None, **how):
    want = br.attention(q, k, v, cu_q, cu_k, dout=dout, **how)
    for name, (value, bound) in want.items():
        br.check(got[name], value, bound, name)


LENS = [
    ([1], [1]), ([128], [128]), ([129], [127]), ([5, 0, 3, 200], [5, 0, 3, 200]), ([1, 1, 1, 1], [300, 1, 64, 7]),
    ([300], [700]), ([40, 70], [0, 13]), ([2, 130, 1, 260, 17], [2, 130, 1, 260, 17]), ([4, 4, 4], [1000, 4, 129]),
    ([385], [1]), ([0, 0, 64], [0, 7, 64]), ([7] * 40, [7] * 40),
]
MASKS = [dict(), dict(causal=True), dict(causal=True, prefix=True), dict(cap=20.0), dict(causal=True, bias=True, cap=5.0)]


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("mask", range(len(MASKS)))
@pytest.mark.parametrize("h,hk,dim,dtype", [(2, 2, 128, BF), (3, 1, 64, FP), (4, 2, 72, BF)])
def test_attention(lens, mask, h, hk, dim, dtype):
    q_lens, k_lens = LENS[lens]
    how = dict(MASKS[mask])
    cu_q, cu_k = ends(q_lens), ends(k_lens)
    tq, tk = cu_q[-1], cu_k[-1]
    if how.pop("prefix", False):
        how["prefix"] = [(n * 2) // 3 + 1 if d % 2 == 0 else 0 for d, n in enumerate(k_lens)]
    if how.pop("bias", False):
        how["slopes"] = 2.0 ** -torch.arange(1, h + 1, device="cuda").float()
    q, k, v = rand((tq, h, dim), dtype, 1, 1.5), rand((tk, hk, dim), dtype, 2, 1.5), rand((tk, hk, dim), dtype, 3)
    dout = rand((tq, h, dim), dtype, 4)
    got = attend(q, k, v, cu_q, cu_k, dout, **how)
    against_reference(got, q, k, v, cu_q, cu_k, dout, **how)


@pytest.mark.parametrize("h,hk,dim,dtype", [(1, 1, 8, BF), (8, 1, 16, FP), (5, 5, 40, BF), (16, 2, 96, FP), (6, 2, 128, FP),
                                            (10, 2, 104, BF)])
def test_attention_head_layouts(h, hk, dim, dtype):
    cu_q, cu_k = [0, 150, 190, 450], [0, 150, 290, 450]
    q, k, v = rand((450, h, dim), dtype, 1), rand((450, hk, dim), dtype, 2), rand((450, hk, dim), dtype, 3)
    dout = rand((450, h, dim), dtype, 4)
    for how in (dict(), dict(causal=True, scale=0.3)):
        got = attend(q, k, v, cu_q, cu_k, dout, **how)
        against_reference(got, q, k, v, cu_q, cu_k, dout, **how)


@pytest.mark.parametrize("h,hk,dim", [(32, 8, 128), (8, 8, 64), (6, 1, 128), (16, 1, 80)])
@pytest.mark.parametrize("new", [1, 2, 4])
def test_attention_of_new_tokens_over_a_long_cache(h, hk, dim, new):
    k_lens = [5000, new, 777, 1, 2049, 0]
    cu_q, cu_k = ends([new] * len(k_lens)), ends(k_lens)
    q, k, v = rand((cu_q[-1], h, dim), BF, 1, 1.5), rand((cu_k[-1], hk, dim), BF, 2, 1.5), rand((cu_k[-1], hk, dim), BF, 3)
    for how in (dict(causal=True), dict(cap=30.0, slopes=torch.full((h,), 0.01, device="cuda"))):
        got = attend(q, k, v, cu_q, cu_k, **how)
        against_reference(got, q, k, v, cu_q, cu_k, **how)


def test_attention_strided_inputs():
    """Slices of a fused projection, heads before tokens, rows of a wider cache."""
    cu = [0, 100, 333]
    qkv = rand((333, 8, 64), BF, 1)
    heads_first = rand((4, 333, 64), BF, 2).transpose(0, 1)
    wide = rand((333, 2, 200), BF, 3)[..., 8:72]
    dout = rand((333, 4, 128), BF, 4)[..., 64:]
    for q, k, v in ((qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]), (heads_first, wide, qkv[:, 2:4])):
        got = attend(q, k, v, cu, cu, dout, causal=True)
        against_reference(got, q, k, v, cu, cu, dout, causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_ignores_what_it_does_not_see(causal, dim):
    """NaN and infinities in tokens of no document, in other documents and (in
    single-query documents) in later keys reach nothing that does not see them."""
    cu_q, cu_k = [3, 60, 261, 300], [5, 90, 291, 330]
    shape = dict(q=(310, 2, dim), k=(340, 1, dim), v=(340, 1, dim), dout=(310, 2, dim))
    t = {n: rand(s, BF, i) for i, (n, s) in enumerate(shape.items())}
    clean = attend(t["q"], t["k"], t["v"], cu_q, cu_k, t["dout"], causal=causal)
    against_reference(clean, t["q"], t["k"], t["v"], cu_q, cu_k, t["dout"], causal=causal)
    bad = {n: x.clone() for n, x in t.items()}
    for n, doc, outside in (("q", (60, 261), [(0, 3), (300, 310)]), ("dout", (60, 261), [(0, 3), (300, 310)]),
                            ("k", (90, 291), [(0, 5), (330, 340)]), ("v", (90, 291), [(0, 5), (330, 340)])):
        for lo, hi in outside + [doc]:
            bad[n][lo:hi] = math.nan
            bad[n][lo:hi:2] = math.inf
    got = attend(bad["q"], bad["k"], bad["v"], cu_q, cu_k, bad["dout"], causal=causal)
    for name in got:
        key = name in ("dk", "dv")
        for lo, hi in (((5, 90), (291, 330)) if key else ((3, 60), (261, 300))):
            pick = (lambda x: x[:, lo:hi]) if name == "lse" else (lambda x: x[lo:hi])
            assert torch.equal(pick(got[name]), pick(clean[name])), name
        for lo, hi in (((0, 5), (330, 340)) if key else ((0, 3), (300, 310))):
            if name == "lse":
                assert (got[name][:, lo:hi] == -math.inf).all()
            else:
                assert not got[name][lo:hi].any(), name
    assert torch.isnan(got["out"][60:261]).any()            # and those that see them show it


def test_attention_causal_future_is_not_read():
    """A NaN in a late value row shows in the queries that see it and in no earlier one."""
    n = 300
    q, k, v = (rand((n, 1, 64), FP, s) for s in (1, 2, 3))
    dout = rand((n, 1, 64), FP, 4)
    clean = attend(q, k, v, [0, n], [0, n], dout, causal=True)
    v[200, 0, 5] = math.nan
    got = attend(q, k, v, [0, n], [0, n], dout, causal=True)
    assert torch.equal(got["out"][:200], clean["out"][:200])
    assert torch.isnan(got["out"][200:, 0, 5]).all() and not torch.isnan(got["out"][200:, 0, :5]).any()
    assert torch.equal(got["dq"][:200], clean["dq"][:200]) and torch.isnan(got["dq"][200:]).all()


def test_attention_extreme_scores():
    """Scores far beyond the range of exp, and of -inf."""
    cu = [0, 200]
    q, k, v = rand((200, 1, 64), BF, 1, 60.0), rand((200, 1, 64), BF, 2, 60.0), rand((200, 1, 64), BF, 3)
    dout = rand((200, 1, 64), BF, 4)
    got = attend(q, k, v, cu, cu, dout)
    for t in got.values():
        assert torch.isfinite(t.float()).all()
    against_reference({n: got[n] for n in ("out", "lse")}, q, k, v, cu, cu)
    q1, k1 = torch.zeros_like(q), torch.zeros_like(k)
    q1[..., 0], k1[:100, :, 0] = 1.0, -math.inf             # half of the keys score -inf
    r = attend(q1, k1, v, cu, cu)
    br.check(r["out"][:, 0], v[100:, 0].double().mean(0).expand(200, 64), 2.0 ** -7, "half at -inf")


def test_attention_without_ends_streams_graphs_and_same_bits():
    q, k, v, dout = (rand((500, 4, 128), BF, s) for s in (1, 2, 3, 4))
    got = attend(q, k, v, [0, 500], [0, 500], dout, causal=True)
    out, lse = gn.attention_packed(q, k, v, causal=True)
    assert torch.equal(out, got["out"]) and torch.equal(lse, got["lse"])
    again = attend(q, k, v, [0, 500], [0, 500], dout, causal=True)
    assert all(torch.equal(again[n], got[n]) for n in got)
    # another stream than the current one, its tensors let go at once
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        other = gn.attention_packed(q.clone(), k.clone(), v.clone(), causal=True)[0]
        o, s = gn.attention_packed(q, k, v, causal=True, stream=side)
        g = gn.attention_packed_backward(dout, q, k, v, o, s, causal=True, stream=side)
        del other
    side.synchronize()
    assert torch.equal(o, out) and all(torch.equal(a, got[n]) for a, n in zip(g, ("dq", "dk", "dv")))
    # one capture of forward and backward, replayed on new inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = gn.attention_packed(q, k, v, causal=True)
        g = gn.attention_packed_backward(dout, q, k, v, o, s, causal=True)
    q.copy_(rand(q.shape, BF, 9))
    graph.replay()
    torch.cuda.synchronize()
    want = attend(q, k, v, [0, 500], [0, 500], dout, causal=True)
    assert torch.equal(o, want["out"]) and all(torch.equal(a, want[n]) for a, n in zip(g, ("dq", "dk", "dv")))


def test_attention_bad_ends_are_clamped():
    """Ends out of range or out of order give some result, and stay inside the tensors."""
    q, k, v, dout = (rand((300, 2, 64), BF, s) for s in (1, 2, 3, 4))
    for cu in ([0, 100, 5000], [-50, 100, 300], [0, 200, 100], [400, 500, 600], [2 ** 31 - 1, -2 ** 31, 7]):
        for causal in (False, True):
            attend(q, k, v, cu, cu, dout, causal=causal, prefix=[2 ** 31 - 1, -5] if causal else None)
    out, clean = guarded(q.shape, BF)
    gn.attention_packed(q, k, v, i32([-9, 700]), i32([3, 2 ** 30]), out=out)
    torch.cuda.synchronize()
    clean()


def test_attention_not_supported():
    q, k = rand((10, 4, 64), BF, 1), rand((10, 2, 64), BF, 2)
    cu = i32([0, 10])
    assert gn.attention_packed(q, k, k, cu, cu) is not None
    assert gn.attention_packed(q.float(), k.float(), k.float()) is None
    assert gn.attention_packed(q, k, k.half()) is None
    assert gn.attention_packed(q, k, k[:9]) is None
    assert gn.attention_packed(q[:, :3], k, k) is None
    assert gn.attention_packed(q, k, k, cu, None) is None
    assert gn.attention_packed(q, k, k, cu.long(), cu.long()) is None
    assert gn.attention_packed(q, k, k, cu, i32([0, 5, 10])) is None
    assert gn.attention_packed(q, k, k, cu, cu, prefix=i32([3])) is None
    assert gn.attention_packed(q, k, k, slopes=torch.ones(3, device="cuda")) is None
    assert gn.attention_packed(q.clone().requires_grad_(), k, k) is None
    assert gn.attention_packed(q.transpose(1, 2), k, k) is None
    out, lse = gn.attention_packed(q, k, k)
    assert gn.attention_packed_backward(q, q, k, k, out, lse.t()) is None
    assert gn.attention_packed_backward(q.sum().expand(q.shape), q, k, k, out, lse) is None
    with pytest.warns(UserWarning):
        assert gn.attention_packed(rand((4, 1, 136), BF, 1), rand((4, 1, 136), BF, 1), rand((4, 1, 136), BF, 1)) is None
    with pytest.warns(UserWarning):                          # rows that are not 16-byte aligned
        assert gn.attention_packed(rand((4, 1, 68), BF, 1)[..., 4:], *[rand((4, 1, 64), BF, 1)] * 2) is None
    empty = gn.attention_packed(q[:0], k, k)
    assert empty[0].shape == (0, 4, 64)
    d = gn.attention_packed_backward(q[:0], q[:0], k, k, *empty)
    assert not d[1].any() and not d[2].any()
    out, lse = gn.attention_packed(q, k[:0], k[:0])
    assert not out.any() and (lse == -math.inf).all()
