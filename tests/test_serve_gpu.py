"""RMS norm and the paged cache in 8 bits on the GPU against their definitions in 64
bits (tests/serve_ref.py, which also derives how far each output may be)."""
import math

import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from tests import block_ref as br
from tests import gpu_util as gu
from tests import serve_ref as sr

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


def rand(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype).cuda()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def same(a, b):
    """The same bits (NaN where NaN)."""
    if a.dtype == sr.E4M3:
        return torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return torch.equal(a.nan_to_num(123.0), b.nan_to_num(123.0)) and torch.equal(a.isnan(), b.isnan())


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
def check_rms(x, w, residual, dy, dtotal, eps=1e-3):
    want = sr.rms_norm(x, w, eps, residual, dy, dtotal)
    y, none, total, rstd = gn.rms_norm(x, w, residual=residual, eps=eps)
    assert none is None and (total is x) == (residual is None)
    dx, dw = gn.rms_norm_backward(dy, total, rstd, w, dtotal=dtotal)
    y8, scales, total8, rstd8 = gn.rms_norm(x, w, residual=residual, eps=eps, quantize=True)
    got = dict(y=y, total=total, rstd=rstd, dx=dx, scales=scales, y8=y8.double() * scales.double()[:, None])
    if w is not None:
        got["dw"] = dw
    else:
        assert dw is None
    for name, value in got.items():
        br.check(value, *want[name], f"{name} {tuple(x.shape)}")
    assert same(rstd8, rstd) and same(total8, total)
    return got


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 6144), (5, 8), (257, 128), (1000, 64), (33, 40), (129, 1003),
                                       (2, 16384), (3, 16383), (700, 1536), (19, 5000), (311, 12288), (4099, 16), (7, 4100)])
@pytest.mark.parametrize("weight,residual", [(None, True), ("own", False), (F32, True)])
def test_rms_norm(rows, cols, dtype, weight, residual):
    x, dy, dtotal = (rand((rows, cols), dtype, s, 2.0) for s in (1, 2, 3))
    r = rand((rows, cols), dtype, 4, 3.0) if residual else None
    w = None if weight is None else rand((cols,), dtype if weight == "own" else weight, 5, 0.3) + 1.0
    check_rms(x, w, r, dy, dtotal if residual else None)


@pytest.mark.parametrize("rows,cols,wide,start,dtype", [
    (40001, 128, 160, 8, FP), (9001, 257, 257, 0, F32), (2000, 6144, 6152, 8, BF), (5003, 1001, 1003, 1, BF), (700, 12001, 12001, 0, FP)])
def test_rms_norm_many_rows_out_of_wider_tensors(rows, cols, wide, start, dtype):
    x, r, dy, dt = (rand((rows, wide), dtype, s, 2.0)[:, start:start + cols] for s in (1, 2, 3, 4))
    got = check_rms(x, rand((cols,), F32, 5) + 1.0, r, dy, dt)
    again = check_rms(x, rand((cols,), F32, 5) + 1.0, r, dy, dt)
    assert all(same(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("cols", [32, 128, 351, 352, 6144, 6143, 30])
def test_rms_norm_halves_of_a_step_in_8_bits(cols, dtype):
    """What lies halfway between two e4m3 numbers goes to the even one: t weight is exact here,
    and so is which side of the middle 448 / max of it lies (all else is 2^-11 away from one)."""
    most = torch.tensor([28, 56, 84, 112, 140, 168, 196, 224, 252], dtype=torch.float64)
    gen = torch.Generator().manual_seed(cols)
    x = torch.randint(-252, 253, (most.shape[0], cols), generator=gen).double().clamp(-most[:, None], most[:, None])
    x[:, cols // 2] = most
    q = x * 448 / most[:, None]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    want = torch.round(q / step) * step
    w = torch.full((cols,), 0.75, device="cuda", dtype=dtype)
    for weight in (None, w):
        y, scales, _, rstd = gn.rms_norm(x.to(dtype).cuda(), weight, eps=1e-3, quantize=True)
        assert torch.equal(y.double().cpu(), want)
        by = rstd.double() * (1.0 if weight is None else 0.75) * most.cuda() / 448
        assert ((scales.double() - by).abs() <= 2.0 ** -22 * by).all()


@pytest.mark.parametrize("start", range(8))
@pytest.mark.parametrize("rows,cols,dtype", [
    (777, 64, BF), (2001, 65, FP), (1301, 131, BF), (401, 4101, BF), (333, 8191, FP), (211, 8198, BF), (5, 16384, FP), (1, 71, BF)])
def test_rms_norm_rows_that_begin_at_any_element(rows, cols, dtype, start):
    def shifted(seed):
        wide = rand((rows * cols + start,), dtype, seed, 2.0)
        return wide[start:].view(rows, cols)

    x, r, dy, dt = (shifted(s) for s in (1, 2, 3, 4))
    w = rand((cols,), dtype, 5, 0.3) + 1.0
    want = sr.rms_norm(x, w, 1e-3, r, dy, dt)
    got = {}
    room = {n: torch.full((rows * cols + start + 9,), 7.0, dtype=dtype, device="cuda") for n in ("y", "total", "dx")}
    into = {n: v[start:start + rows * cols].view(rows, cols) for n, v in room.items()}
    bytes_ = torch.full((rows * cols + start + 9,), 99, dtype=torch.uint8, device="cuda")
    y8 = bytes_[start:start + rows * cols].view(rows, cols).view(sr.E4M3)
    for again in range(2):
        _, _, _, rstd = gn.rms_norm(x, w, residual=r, eps=1e-3, out=into["y"], total_out=into["total"])
        _, scales, _, rstd8 = gn.rms_norm(x, w, residual=r, eps=1e-3, out=y8, total_out=into["total"], quantize=True)
        _, dw = gn.rms_norm_backward(dy, into["total"], rstd, w, dtotal=dt, out=into["dx"])
        now = dict(y=into["y"], total=into["total"], rstd=rstd, dx=into["dx"], dw=dw, scales=scales,
                   y8=y8.double() * scales.double()[:, None])
        if again:
            assert all(same(now[n], got[n]) for n in now)
        got = {n: v.clone() for n, v in now.items()}
    for name, value in got.items():
        br.check(value, *want[name], f"{name} {rows}x{cols} from {start}")
    assert same(rstd8, rstd)
    for v in room.values():
        assert (v[:start] == 7.0).all() and (v[start + rows * cols:] == 7.0).all()
    assert (bytes_[:start] == 99).all() and (bytes_[start + rows * cols:] == 99).all()


def test_rms_norm_heads_of_a_projection_and_broadcast_rows():
    qkv = rand((300, 7, 64), BF, 1, 2.0)
    w = rand((64,), BF, 2) + 1.0
    x = qkv[:, 2:6]
    y, _, total, rstd = gn.rms_norm(x, w, eps=1e-5)
    assert y.is_contiguous() and rstd.shape == (300, 4) and total is x
    dy = rand((300, 1, 64), BF, 3).expand(300, 4, 64)
    dx, dw = gn.rms_norm_backward(dy, x, rstd, w)
    flat = lambda t: t.reshape(-1, 64)  # noqa: E731
    want = sr.rms_norm(flat(x), w, 1e-5, dy=flat(dy))
    for name, got in dict(y=flat(y), rstd=rstd.flatten(), dx=flat(dx), dw=dw).items():
        br.check(got, *want[name], name)
    into = torch.full((300, 9, 64), 5.0, dtype=BF, device="cuda")
    out = into[:, 3:7]
    assert gn.rms_norm(x, w, eps=1e-5, out=out)[0] is out and same(out.contiguous(), y)
    assert (into[:, :3] == 5.0).all() and (into[:, 7:] == 5.0).all()


def test_rms_norm_in_place():
    x, r, dy, dt = (rand((77, 1000), BF, s) for s in (1, 2, 3, 4))
    w = rand((1000,), F32, 5) + 1.0
    want = gn.rms_norm(x, w, residual=r)
    stream = r.clone()
    y, _, total, rstd = gn.rms_norm(x, w, residual=stream, total_out=stream)
    assert total is stream and same(y, want[0]) and same(stream, want[2])
    onto = x.clone()
    assert same(gn.rms_norm(onto, w, residual=r, total_out=onto)[0], want[0]) and same(onto, want[2])
    own = x.clone()
    assert same(gn.rms_norm(own, w, out=own)[0], gn.rms_norm(x, w)[0])
    dx, dw = gn.rms_norm_backward(dy, total, rstd, w, dtotal=dt)
    for n in range(3):
        a = [dy.clone(), total.clone(), dt.clone()]
        got = gn.rms_norm_backward(a[0], a[1], rstd, w, dtotal=a[2], out=a[n])
        assert got[0] is a[n] and same(got[0], dx) and same(got[1], dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [71, 1001, 9001])
def test_rms_norm_in_place_in_odd_widths(cols, dtype):
    x, r, dy, dt = (rand((777, cols), dtype, s) for s in (1, 2, 3, 4))
    w = rand((cols,), F32, 5) + 1.0
    want = gn.rms_norm(x, w, residual=r)
    for onto in (r.clone(), x.clone()):
        a, b = (x, onto) if same(onto, r) else (onto, r)
        y, _, total, rstd = gn.rms_norm(a, w, residual=b, total_out=onto)
        assert total is onto and same(y, want[0]) and same(onto, want[2]) and same(rstd, want[3])
    own = x.clone()
    assert same(gn.rms_norm(own, w, out=own)[0], gn.rms_norm(x, w)[0])
    dx, dw = gn.rms_norm_backward(dy, total, rstd, w, dtotal=dt)
    for n in range(3):
        a = [dy.clone(), total.clone(), dt.clone()]
        got = gn.rms_norm_backward(a[0], a[1], rstd, w, dtotal=a[2], out=a[n])
        assert got[0] is a[n] and same(got[0], dx) and same(got[1], dw)


def test_rms_norm_rows_of_zeros_nan_and_infinity():
    x = rand((6, 64), F32, 1)
    x[1] = 0.0
    x[2, 5] = math.nan
    x[3, 7] = math.inf
    x[4] *= 1e-36
    y, scales, _, rstd = gn.rms_norm(x, eps=1e-6, quantize=True)
    clean = gn.rms_norm(x[[0, 5]].contiguous(), eps=1e-6, quantize=True)
    assert same(y[[0, 5]], clean[0]) and same(scales[[0, 5]], clean[1])
    v = y.float()
    assert scales[1] == 0 and not v[1].any() and scales[4] == 0 and not v[4].any()
    assert scales[2:4].isnan().all() and v[2].isnan().all()
    assert rstd[3] == 0 and rstd[2].isnan()


def test_rms_norm_nothing_and_not_supported():
    x = rand((4, 64), BF, 1)
    w = rand((64,), F32, 2)
    y, _, _, rstd = gn.rms_norm(x[:0], w)
    assert y.shape == (0, 64)
    dx, dw = gn.rms_norm_backward(x[:0], x[:0], rstd, w)
    assert dx.shape == (0, 64) and not dw.any()
    assert gn.rms_norm(x.double()) is None and gn.rms_norm(x, w[:32]) is None
    assert gn.rms_norm(x, residual=x.float()) is None and gn.rms_norm(x, total_out=x) is None
    assert gn.rms_norm(x.t()) is None and gn.rms_norm(x.clone().requires_grad_()) is None
    assert gn.rms_norm(x, quantize=True, out=torch.empty_like(x)) is None
    assert gn.rms_norm_backward(x, x, rstd, w) is None
    with pytest.warns(UserWarning):
        assert gn.rms_norm(x, eps=math.nan) is None
    with pytest.warns(UserWarning):
        assert gn.rms_norm(x[:2], out=x[1:3]) is None


@pytest.mark.parametrize("rows,cols,dtype", [(600, 2048, BF), (9000, 64, FP), (300, 77, F32)])
def test_rms_norm_outputs_in_bytes_that_lie_anywhere_and_captured(rows, cols, dtype):
    x, w = rand((rows, cols), dtype, 1, 2.0), rand((cols,), dtype, 2) + 1.0
    y, scales, _, rstd = gn.rms_norm(x, w, quantize=True)
    buf = torch.full((rows, cols + 9), 0x11, dtype=torch.uint8, device="cuda")
    into = buf[:, 3:3 + cols].view(sr.E4M3)
    got = gn.rms_norm(x, w, quantize=True, out=into)
    # (single bytes are another kernel's work, whose sums may be a rounding off)
    want = sr.rms_norm(x, w, 1e-6)
    assert got[0] is into
    br.check(into.double() * got[1].double()[:, None], *want["y8"], "bytes")
    br.check(got[1], *want["scales"], "scales")
    assert (buf[:, :3] == 0x11).all() and (buf[:, 3 + cols:] == 0x11).all()
    dy = rand((rows, cols), dtype, 3)
    dx, dw = gn.rms_norm_backward(dy, x, rstd, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = gn.rms_norm(x, w, quantize=True)
        b = gn.rms_norm_backward(dy, x, a[3], w)
    x.neg_()
    graph.replay()
    assert same(a[1], scales) and same(a[3], rstd) and same(a[0].float(), -y.float()) and same(b[1], -dw)


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------
def append_and_check(cache, new, hk, dim, axes=(), theta=1e4, interleaved=True, dtype=BF, heads=0, seed=0, cu=True, pad=(0, 0),
                     positions=None, scale=1.0):
    """`cache` holds its tokens already; the last new[s] of each sequence are written anew."""
    tokens = sum(new) + sum(pad)
    qkv = rand((tokens, heads + 2 * hk, dim), dtype, seed + 1, 1.5 * scale)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:]
    begins = [pad[0]]
    for n in new:
        begins.append(begins[-1] + n)
    if axes and positions is None:
        positions = torch.randint(-5, 4000, (tokens, len(axes)), dtype=torch.int32, device="cuda",
                                  generator=torch.Generator("cuda").manual_seed(seed))
    before = cache.copy()
    how = dict(positions=positions, axes_dim=axes, theta=theta, interleaved=interleaved) if axes else {}
    got = gn.cache_append(k, v, *cache.args(), i32(begins) if cu else None, q=q if heads else None, **how)
    torch.cuda.synchronize()
    assert got is not None
    turned = {}
    for name, x in (("q", q), ("k", k)):
        turned[name] = br.rope(x.float(), positions, axes, theta, interleaved, False) if axes and x.shape[1] else (x.double(), 0.0 * x.double())
    if heads:
        value, bound = br.rope(q, positions, axes, theta, interleaved, False) if axes else (q.double(), 0.0 * q.double())
        br.check(got, value, bound, "q")
    else:
        assert got is True
    touched = set()
    for s, (n, length) in enumerate(zip(new, cache.lens)):
        begin = max(length - n, 0)
        for p in range(begin // cache.page, (length + cache.page - 1) // cache.page if n else 0):
            at = cache.table_host[s][p]
            lo, hi = max(begin, p * cache.page), min(length, (p + 1) * cache.page)
            slot, first = lo - p * cache.page, begins[s] + lo - (length - n)
            touched.add(at)
            for name in "kv":
                x, off = turned["k"] if name == "k" else (v.double(), 0.0 * v.double())
                x, off = x[first:first + hi - lo], off[first:first + hi - lo]
                old, now = before.scales(name)[at].double(), cache.scales(name)[at].double()
                for h in range(hk):
                    most, slack = float(x[:, h].abs().max()), float(off[:, h].max())
                    wants = {max(sr.least_scale(m), float(old[h]) if slot else 0.0) for m in (most, most - slack, most + slack)}
                    assert float(now[h]) in wants, (name, s, p, h, float(now[h]), wants)
                page, was = cache.pages(name)[at], before.pages(name)[at]
                values = page[slot:slot + hi - lo].view(sr.E4M3).double() * now[:, None]
                br.check(values, x, off + 2.0 ** -4 * x.abs() + (2.0 ** -10 * now)[:, None], f"{name} page {p} of {s}")
                if name == "v":                              # nothing turned: the same bytes
                    assert torch.equal(page[slot:slot + hi - lo].view(sr.E4M3).double(), sr.cast_e4m3(x / now[:, None]))
                held = sr.cast_e4m3(was[:slot].view(sr.E4M3).double() * (old / now)[:, None])
                assert torch.equal(page[:slot].view(sr.E4M3).double(), held), (name, s, p)
                assert torch.equal(page[hi - p * cache.page:], was[hi - p * cache.page:])
    for name in "kv":
        keep = [p for p in range(cache.pages(name).shape[0]) if p not in touched]
        assert torch.equal(cache.pages(name)[keep], before.pages(name)[keep])
        assert same(cache.scales(name)[keep], before.scales(name)[keep])


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("page,dim,axes,interleaved", [
    (8, 16, (16,), True), (16, 64, (16, 24, 24), False), (64, 128, (32, 32, 32, 32), True), (64, 128, (16, 56, 56), False),
    (24, 80, (10, 6), True), (256, 96, (22, 22), False), (128, 112, (), True), (40, 48, (6, 4, 2), False)])
def test_append(page, dim, axes, interleaved, dtype):
    new = [1, page, 0, 3, 2 * page + 5, 17]
    lens = [1, page, 5, page + 2, 3 * page + 1, 2 * page]
    for order, heads in (("heads", 6), ("tokens", 0), ("slots", 3)):
        cache = sr.Cache(lens, page, 3, dim, seed=page, order=order)
        append_and_check(cache, new, 3, dim, axes, 2000.0, interleaved, dtype, heads, seed=dim, pad=(2, 3))


@pytest.mark.parametrize("count", [1, 2, 31, 33, 700])
def test_append_one_token_each(count):
    lens = [1 + (37 * n) % 300 for n in range(count)]
    cache = sr.Cache(lens, 32, 2, 64, seed=1)
    append_and_check(cache, [1] * count, 2, 64, (32, 32), heads=8, cu=False)
    append_and_check(cache, [1] * count, 2, 64, (32, 32), heads=8, cu=True, seed=5, scale=40.0)     # scales grow
    append_and_check(cache, [1] * count, 2, 64, (32, 32), heads=1, cu=True, seed=6, scale=1e-3)     # and stay


@pytest.mark.parametrize("kind", [torch.int32, torch.int64, torch.float32])
def test_append_far_positions(kind):
    tokens = 40
    at = torch.tensor([0, 1, -1, 2 ** 20, 123456789, -98765432, 2 ** 31 - 1, -(2 ** 31)] * 5)
    at = at.to(kind) if kind != torch.float32 else at.float() / 3 - 1e-9
    positions = torch.stack([at, at.flip(0)], 1).cuda()
    cache = sr.Cache([tokens], 16, 1, 64, seed=3)
    append_and_check(cache, [tokens], 1, 64, (30, 34), 500.0, True, F32, 2, positions=positions)


def test_append_values_that_are_no_numbers():
    """An infinity or a NaN makes its page and head read as NaN, and nothing else."""
    cache = sr.Cache([100, 40], 32, 2, 32, seed=1)
    clean = cache.copy()
    k, v = rand((20, 2, 32), BF, 1), rand((20, 2, 32), BF, 2)
    cu = i32([0, 10, 20])
    assert gn.cache_append(k, v, *clean.args(), cu) is True
    k[9, 1, 3], v[12, 0, 0] = math.nan, -math.inf
    assert gn.cache_append(k, v, *cache.args(), cu) is True
    for name, s, place, head in (("k", 0, 99, 1), ("v", 1, 32, 0)):
        at = cache.table_host[s][place // 32]
        assert cache.scales(name)[at, head].isnan() and not clean.scales(name)[at, head].isnan()
        cache.scales(name)[at, head] = clean.scales(name)[at, head]
        new = slice(96 % 32, 100 % 32) if s == 0 else slice(32 % 32, 40 % 32)
        assert not cache.pages(name)[at, new, head].any()
        cache.pages(name)[at, :, head] = clean.pages(name)[at, :, head]
    for name in "kv":
        assert torch.equal(cache.pages(name), clean.pages(name)) and same(cache.scales(name), clean.scales(name))
    # a page that reads as NaN stays so until it starts anew
    at = cache.table_host[1][1]
    cache.scales("v")[at, 1] = math.nan
    assert gn.cache_append(k[:1], v[:1], *cache.args(), i32([0, 0, 1])) is True
    assert cache.scales("v")[at, 1].isnan()


def test_append_tiny_and_huge_values():
    for size in (0.0, 1e-38, 1e-30, 1e-10, 1e30, 3e38):
        cache = sr.Cache([64], 32, 2, 32, seed=1)
        k = rand((64, 2, 32), F32, 1).clamp(-0.9, 0.9) * size
        assert gn.cache_append(k, k, *cache.args()) is True
        got = cache.values("k", 0)
        scale = max(2.0 ** -100, size / 448 * 2)
        br.check(got, k.double(), 2.0 ** -4 * k.double().abs() + 2.0 ** -10 * scale, size)


def test_append_bad_tables_lengths_and_ends():
    """Out of range, negative, out of order: some result, nothing outside the tensors."""
    k, v = rand((50, 2, 32), BF, 1), rand((50, 2, 32), BF, 2)
    q = rand((50, 4, 32), BF, 3)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")[:, None]
    for cu in ([0, 20, 5000], [-50, 10, 50], [0, 40, 10], [60, 70, 80], [2 ** 31 - 1, -2 ** 31, 7], [10, 10, 10]):
        for lens in ([-5, 2 ** 31 - 1], [3, 4], [0, 0], [10000, -2 ** 31]):
            for pages in ([-1, 10 ** 9], [2 ** 31 - 1, -2 ** 31]):
                cache = sr.Cache([60, 60], 32, 2, 32, seed=1)
                before = cache.copy()
                cache.lengths = i32(lens)
                cache.table = i32([pages, pages])
                got = gn.cache_append(k, v, *cache.args(), i32(cu), q=q, positions=pos, axes_dim=(32,))
                torch.cuda.synchronize()
                value, bound = br.rope(q, pos, (32,), 1e4, True, False)
                br.check(got, value, bound, "q of every token, stored or not") if sorted(cu) == cu else None
                for name in "kv":
                    assert torch.equal(cache.pages(name), before.pages(name)) and same(cache.scales(name), before.scales(name))


@pytest.mark.parametrize("new", [1, 12, 90])
def test_lengths_past_the_table(new):
    """Tokens past the table are dropped, and nothing moves in their place: what is there
    stays, and the queries see what the table holds."""
    cache = sr.Cache([64, 40], 32, 2, 32, seed=1, width=2)
    before = cache.copy()
    k, v = rand((2 * new, 2, 32), BF, 1), rand((2 * new, 2, 32), BF, 2)
    q = rand((2 * new, 4, 32), BF, 3)
    lengths = i32([64 + new, 64 + new])                     # all new tokens of both lie behind the table
    args = (*cache.args()[:5], lengths)
    assert gn.cache_append(k, v, *args) is True
    for name in "kv":
        assert torch.equal(cache.pages(name), before.pages(name)) and same(cache.scales(name), before.scales(name))
    out, lse = gn.attention_cached(q, *args)
    want = sr.attention(q[:new].contiguous(), sr_first(cache), [0, new], causal=False)
    br.check(out[:new], *want["out"], "out")
    br.check(lse[:, :new], *want["lse"], "lse")


def sr_first(cache):
    """The cache with its first sequence alone."""
    one = cache.copy()
    one.lens, one.table_host = cache.lens[:1], cache.table_host[:1]
    return one


def test_append_layouts_of_one_buffer():
    """Keys and values side by side in one buffer, at every level; q in place."""
    for shape, pick in (((9, 2, 16, 3, 32), lambda b, n: b[:, n]), ((9, 16, 2, 3, 32), lambda b, n: b[:, :, n]),
                        ((9, 16, 3, 2, 32), lambda b, n: b[:, :, :, n]), ((2, 9, 16, 3, 32), lambda b, n: b[n])):
        cache = sr.Cache([70, 30], 16, 3, 32, seed=1, order="tokens")
        buf = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda")
        for n, name in enumerate("kv"):
            part = pick(buf, n)
            part.copy_(cache.pages(name))
            setattr(cache, name + "_bytes", part)
            setattr(cache, name + "_pages", part.view(sr.E4M3))
        append_and_check(cache, [9, 30], 3, 32, (32,), heads=2)
    qkv = rand((10, 6, 32), BF, 1)
    cache = sr.Cache([10], 16, 2, 32)
    want = gn.cache_append(qkv[:, 2:4], qkv[:, 4:], *cache.args(), q=qkv[:, :2], positions=torch.ones(10, 1, device="cuda"), axes_dim=(32,))
    got = gn.cache_append(qkv[:, 2:4], qkv[:, 4:], *cache.args(), q=qkv[:, :2], out=qkv[:, :2],
                          positions=torch.ones(10, 1, device="cuda"), axes_dim=(32,))
    assert same(got.contiguous(), want) and got.data_ptr() == qkv.data_ptr()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend_and_check(cache, new, h, dim, dtype=BF, seed=0, cu=None, size=1.5, **how):
    begins = [0]
    for n in new:
        begins.append(begins[-1] + n)
    q = rand((begins[-1], h, dim), dtype, seed + 1, size)
    out, lse = gn.attention_cached(q, *cache.args(), i32(begins) if cu is None else cu, **how)
    torch.cuda.synchronize()
    want = sr.attention(q, cache, begins, **how)
    br.check(out, *want["out"], f"out {new} {how}")
    br.check(lse, *want["lse"], f"lse {new} {how}")
    return q, out, lse


HEADS = [(1, 1), (4, 4), (8, 2), (16, 2), (7, 1), (40, 1), (20, 4)]


@pytest.mark.parametrize("h,hk", HEADS)
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16), (16, 8), (96, 24), (80, 256), (112, 40)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_one_token_each(h, hk, dim, page, dtype):
    lens = [1, 700, 129, 128, 0, 17, 2 * page, 333]
    cache = sr.Cache(lens, page, hk, dim, seed=dim)
    q, out, lse = attend_and_check(cache, [1] * len(lens), h, dim, dtype)
    again = gn.attention_cached(q, *cache.args())
    assert same(again[0], out) and same(again[1], lse)
    assert not out[4].any() and (lse[:, 4] == -math.inf).all()


@pytest.mark.parametrize("h,hk", HEADS)
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16), (80, 24)])
@pytest.mark.parametrize("how", [dict(), dict(causal=False), dict(cap=5.0), dict(slopes=0.02), dict(cap=20.0, slopes=0.01, scale=-0.2)])
def test_attention_some_tokens_each(h, hk, dim, page, how):
    lens = [5, 700, 129, 40, 3, 0, 300]
    new = [5, 4, 17, 0, 1, 0, 70]
    how = dict(how)
    if "slopes" in how:
        how["slopes"] = torch.full((h,), how["slopes"], device="cuda") * torch.arange(1, h + 1, device="cuda")
    for order in ("heads", "tokens"):
        cache = sr.Cache(lens, page, hk, dim, seed=dim, order=order)
        attend_and_check(cache, new, h, dim, BF if h % 2 else FP, **how)


@pytest.mark.parametrize("h,hk,dim,page,new,lens", [
    (8, 2, 128, 64, [300, 1000], [300, 2500]), (4, 4, 64, 16, [513], [3000]), (16, 1, 96, 32, [257, 3, 64], [900, 1200, 64]),
    (8, 8, 128, 128, [1024], [1024]), (3, 1, 80, 8, [400], [401]), (5, 5, 112, 256, [129, 255], [4000, 255])])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_many_tokens(h, hk, dim, page, new, lens, dtype):
    cache = sr.Cache(lens, page, hk, dim, seed=dim)
    q, out, lse = attend_and_check(cache, new, h, dim, dtype)
    begins = i32([0] + [sum(new[:n + 1]) for n in range(len(new))])
    again = gn.attention_cached(q, *cache.args(), begins)
    assert same(again[0], out) and same(again[1], lse)
    attend_and_check(cache, new, h, dim, dtype, causal=False, cap=10.0)
    attend_and_check(cache, new, h, dim, dtype, slopes=torch.full((h,), 0.02, device="cuda"))


def test_attention_many_sequences():
    lens = [(n * 37) % 260 for n in range(1500)]
    cache = sr.Cache(lens, 32, 1, 32, seed=1)
    attend_and_check(cache, [1] * 1500, 4, 32)
    attend_and_check(cache, [n % 3 for n in range(1500)], 2, 32)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("h,hk,dim,page,new,lens", [
    (8, 2, 128, 64, [300, 1, 1, 8, 9, 0, 1], [300, 2000, 5, 8, 700, 40, 0]), (4, 4, 64, 16, [1, 32, 33, 1, 200], [900, 32, 3000, 1, 200]),
    (16, 1, 96, 32, [2, 3, 1, 1, 40], [800, 900, 1, 130, 41]), (32, 1, 80, 24, [1, 2, 1, 7], [500, 600, 3, 7]),
    (33, 1, 48, 8, [1, 2, 1], [100, 300, 0]), (64, 8, 128, 256, [4, 5, 1, 1, 70], [4, 3000, 1500, 257, 900]),
    (16, 2, 112, 40, [0, 0, 500], [10, 0, 900]), (16, 2, 112, 40, [1] * 20 + [4], [100] * 21)])
def test_attention_single_tokens_beside_long_runs(h, hk, dim, page, new, lens, dtype):
    """Few tokens and many of them in one call, with tokens of no sequence around them."""
    cache = sr.Cache(lens, page, hk, dim, seed=dim)
    ahead, behind = 37, 5
    begins = [0]
    for n in new:
        begins.append(begins[-1] + n)
    q = rand((ahead + begins[-1] + behind, h, dim), dtype, 3, 1.5)
    inside = slice(ahead, ahead + begins[-1])
    cu = i32([ahead + n for n in begins])
    for how in (dict(), dict(causal=False, cap=7.0), dict(slopes=torch.full((h,), 0.03, device="cuda"))):
        out, lse = gn.attention_cached(q, *cache.args(), cu, **how)
        again = gn.attention_cached(q, *cache.args(), cu, **how)
        want = sr.attention(q[inside].contiguous(), cache, begins, **how)
        br.check(out[inside], *want["out"], f"out {new} {how}")
        br.check(lse[:, inside], *want["lse"], f"lse {new} {how}")
        assert same(again[0], out) and same(again[1], lse)
        for gone in (slice(0, ahead), slice(ahead + begins[-1], None)):
            assert not out[gone].any() and (lse[:, gone] == -math.inf).all()


def test_attention_captured_once_for_any_counts():
    """The counts of new tokens are the device's: a captured call follows them."""
    cache = sr.Cache([300, 900, 40, 5], 32, 2, 64, seed=1)
    q = rand((240, 8, 64), BF, 1, 1.5)
    cu = i32([0, 60, 120, 160, 165])
    gn.attention_cached(q, *cache.args(), cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = gn.attention_cached(q, *cache.args(), cu)
    for begins in ([0, 1, 2, 3, 4], [0, 200, 201, 240, 240], [10, 18, 27, 27, 28], [0, 0, 0, 40, 45], [0, 60, 120, 160, 165]):
        cu.copy_(i32(begins))
        for again in range(2):
            out.fill_(9.0)
            lse.fill_(9.0)
            graph.replay()
        eager = gn.attention_cached(q, *cache.args(), i32(begins))
        assert same(out, eager[0]) and same(lse, eager[1])
        inside = slice(begins[0], begins[-1])
        want = sr.attention(q[inside].contiguous(), cache, [b - begins[0] for b in begins])
        br.check(out[inside], *want["out"], f"out {begins}")
        br.check(lse[:, inside], *want["lse"], f"lse {begins}")


def test_attention_padded_batch():
    """Tokens ahead of the first sequence and behind the last, sequences without tokens."""
    cache = sr.Cache([50, 60, 7, 0], 16, 2, 64, seed=1)
    q = rand((30, 4, 64), BF, 1)
    out, lse = gn.attention_cached(q, *cache.args(), i32([3, 10, 20, 20, 24]))
    want = sr.attention(q[3:24].contiguous(), cache, [0, 7, 17, 17, 21])
    br.check(out[3:24], *want["out"], "out")
    br.check(lse[:, 3:24], *want["lse"], "lse")
    for gone in (slice(0, 3), slice(20, 30)):
        assert not out[gone].any() and (lse[:, gone] == -math.inf).all()


def test_attention_more_new_tokens_than_the_cache_holds():
    cache = sr.Cache([5, 3], 16, 1, 32, seed=1)
    attend_and_check(cache, [9, 40], 2, 32)


@pytest.mark.parametrize("new", [1, 3, 200])
def test_attention_ignores_what_it_does_not_see(new):
    """NaN bytes and scales in unowned pages and slots do nothing (a Cache holds them
    everywhere); a page of NaN scale shows in the queries that see it and no others."""
    lens = [max(new, 70), 300, 500]
    cache = sr.Cache(lens, 32, 2, 64, seed=1)
    q, out, lse = attend_and_check(cache, [new] * 3, 4, 64)
    cu = i32([0, new, 2 * new, 3 * new])
    for name in "kv":
        bad = cache.copy()
        bad.scales(name)[cache.table_host[1][299 // 32], 0] = math.nan      # the page of places 288 on
        got, got_lse = gn.attention_cached(q, *bad.args(), cu)
        sees = new + max(0, 300 - 12 - new), slice(2 * new - min(new, 12), 2 * new)
        rows = sees[1]
        assert got[rows, :2].isnan().all() and (name == "v" or got_lse[:2, rows].isnan().all())
        keep = torch.ones(3 * new, dtype=torch.bool, device="cuda")
        keep[rows] = False
        assert same(got[keep], out[keep]) and same(got[:, 2:], out[:, 2:])
        assert same(got_lse[:, keep], lse[:, keep]) and same(got_lse[2:], lse[2:])


def test_attention_of_a_query_that_is_no_number():
    cache = sr.Cache([100, 200], 32, 1, 64, seed=1)
    for new in (2, 70):
        q, out, lse = attend_and_check(cache, [new, new], 4, 64)
        cu = i32([0, new, 2 * new])
        bad = q.clone()
        bad[1, 2, 5], bad[new + 1, 0, 0] = math.nan, math.inf
        got, got_lse = gn.attention_cached(bad, *cache.args(), cu)
        for t, h in ((1, 2), (new + 1, 0)):
            assert got[t, h].isnan().all() and got_lse[h, t].isnan()
            got[t, h], got_lse[h, t] = out[t, h], lse[h, t]
        assert same(got, out) and same(got_lse, lse)


@pytest.mark.parametrize("new", [1, 64])
def test_attention_extreme_scales_and_scores(new):
    cache = sr.Cache([300], 32, 1, 64, seed=1)
    q, _, _ = attend_and_check(cache, [new], 2, 64, size=40.0)              # scores far beyond exp's range
    for name, factor in (("v", 2.0 ** -60), ("v", 2.0 ** 60), ("k", 2.0 ** -60), ("v", 0.0)):
        other = cache.copy()
        other.scales(name).mul_(factor)
        out, lse = gn.attention_cached(q, *other.args())
        want = sr.attention(q, other, [0, new])
        for got, (value, bound) in ((out, want["out"]), (lse, want["lse"])):
            br.check(got, value, bound + (1e-25 if factor == 0 else 0), (name, factor))
    # pages of very different scales, zeros among them
    other = cache.copy()
    other.v_scales.mul_(torch.exp2(torch.arange(other.v_scales.shape[0], device="cuda").float() * 9 - 40)[:, None])
    other.v_scales[cache.table_host[0][3]] = 0.0
    out, _ = gn.attention_cached(q, *other.args())
    br.check(out, *sr.attention(q, other, [0, new])["out"], "scales")


def test_attention_sink_and_many_small_weights():
    """One key far above the others, whose sum still is most of the weight."""
    cache = sr.Cache([4096], 64, 1, 64, seed=1, spread=0.0)
    cache.scales("k")[cache.table_host[0][0]] *= 4
    for new in (1, 200):
        attend_and_check(cache, [new], 4, 64, size=0.3)
        attend_and_check(cache, [new], 4, 64, FP, size=0.3)


def test_attention_slices_streams_graphs_and_bad_tables():
    cache = sr.Cache([90, 260, 33], 32, 2, 64, seed=1)
    wide = rand((6, 9, 80), BF, 1)
    q = wide[:, 1:5, 8:72]
    cu = i32([0, 1, 5, 6])
    want = gn.attention_cached(q.contiguous(), *cache.args(), cu)
    got = gn.attention_cached(q, *cache.args(), cu)
    assert same(got[0], want[0]) and same(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        other = gn.attention_cached(q.clone(), *cache.args(), cu)
        got = gn.attention_cached(q, *cache.args(), cu, stream=side)
        del other
    side.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])
    # two graphs, replayed by turns on inputs that change
    q, graphs, outs = q.clone(), [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(gn.attention_cached(q, *cache.args(), cu))
        graphs.append(graph)
    for seed in (5, 6):
        q.copy_(rand(q.shape, BF, seed))
        for graph in graphs:
            graph.replay()
        want = gn.attention_cached(q, *cache.args(), cu)
        assert all(same(o[0], want[0]) and same(o[1], want[1]) for o in outs)
    for bad_cu in ([0, 100, 5000, 6], [-50, 2, 1, 6], [2 ** 31 - 1, -2 ** 31, 7, 8]):
        for lens in ([-5, 2 ** 31 - 1, 80], [10000, -2 ** 31, 3]):
            gn.attention_cached(q, cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales,
                                i32([[-1] * 9, [10 ** 9] * 9, [2 ** 31 - 1, -2 ** 31] + [0] * 7]), i32(lens), i32(bad_cu))
            torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_append_then_attend_like_packed_attention_of_the_rounded_keys():
    """Prompts in chunks, then single tokens, against attention_packed of what the cache holds."""
    h, hk, dim, page = 8, 2, 64, 32
    chunks = [[100, 40], [33, 1], [1, 1], [1, 1], [0, 65]]
    cache = sr.Cache([0, 0], page, hk, dim, seed=1, spare=12, width=6)
    order = torch.randperm(12, generator=torch.Generator().manual_seed(2)).view(2, 6)
    cache.table_host, cache.table = order.tolist(), order.int().cuda()
    lens = [0, 0]
    for step, new in enumerate(chunks):
        lens = [a + b for a, b in zip(lens, new)]
        cache.lens, cache.lengths = lens, i32(lens)
        tokens = sum(new)
        qkv = rand((tokens, h + 2 * hk, dim), BF, step, 1.5)
        positions = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)])[:, None].int().cuda()
        cu = i32([0, new[0], tokens])
        q = gn.cache_append(qkv[:, h:h + hk], qkv[:, h + hk:], *cache.args(), cu, q=qkv[:, :h], positions=positions, axes_dim=(64,))
        out, lse = gn.attention_cached(q, *cache.args(), cu)
        want = sr.attention(q, cache, [0, new[0], tokens])
        br.check(out, *want["out"], f"out {step}")
        br.check(lse, *want["lse"], f"lse {step}")
        k, v = (torch.cat([cache.values(n, s) for s in range(2)]).to(BF) for n in "kv")     # exact in bf16
        packed = gn.attention_packed(q, k, v, cu, i32([0, lens[0], sum(lens)]), causal=True)
        br.check(packed[0], want["out"][0], 2 * want["out"][1] + 2.0 ** -6 * want["out"][0].abs().amax(), f"packed {step}")


def test_append_and_attention_not_supported():
    cache = sr.Cache([20, 30], 16, 2, 32, seed=1)
    q, k = rand((4, 4, 32), BF, 1), rand((4, 2, 32), BF, 2)
    a = cache.args()
    assert gn.attention_cached(q, *a) is not None and gn.cache_append(k, k, *a) is True
    swap = lambda n, t: a[:n] + (t,) + a[n + 1:]  # noqa: E731
    for bad in (swap(0, cache.k_bytes), swap(1, cache.v_pages[:, :, :1]), swap(2, a[2].double()), swap(3, a[3].t()),
                swap(4, a[4].long()), swap(4, a[4][0]), swap(5, a[5][:1]), swap(0, a[0].cpu())):
        assert gn.attention_cached(q, *bad) is None
        assert gn.cache_append(k, k, *bad) is None
    assert gn.attention_cached(q.float(), *a) is None and gn.attention_cached(q[..., :16], *a) is None
    assert gn.attention_cached(q, *a, i32([0, 4])) is None and gn.attention_cached(q, *a, scale=math.inf) is None
    assert gn.attention_cached(q.clone().requires_grad_(), *a) is None
    assert gn.cache_append(k, k[:3], *a) is None and gn.cache_append(k[:, :1], k[:, :1], *a) is None
    assert gn.cache_append(k, k, *a, q=q.half()) is None and gn.cache_append(k, k, *a, axes_dim=(32,)) is None
    assert gn.cache_append(k, k, *a, positions=torch.zeros(4, 1, device="cuda")) is None
    assert gn.cache_append(k, k, *a, out=q) is None
    assert gn.attention_cached(q[:0], *a)[0].shape == (0, 4, 32) and gn.cache_append(k[:0], k[:0], *a) is True
    one = torch.zeros(32, device="cuda", dtype=torch.uint8).expand(5, 16, 2, 32).view(sr.E4M3)
    for call in (lambda: gn.attention_cached(q[:3], *a), lambda: gn.cache_append(k[:3], k[:3], *a),
                 lambda: gn.attention_cached(q[:, :3], *a), lambda: gn.attention_cached(q, *a, cap=-1.0),
                 lambda: gn.cache_append(k, k, *a, positions=torch.zeros(4, 1, device="cuda"), axes_dim=(34,)),
                 lambda: gn.cache_append(k, k, *a, positions=torch.zeros(4, 1, device="cuda"), axes_dim=(32,), theta=0.0),
                 lambda: gn.cache_append(k, k, a[0], a[0], *a[2:]), lambda: gn.cache_append(k, k, a[0], a[1], a[2], a[2], *a[4:]),
                 lambda: gn.cache_append(k, k, one, one, *(torch.ones(5, 2, device="cuda") for _ in range(2)), *a[4:])):
        with pytest.warns(UserWarning):
            assert call() is None
