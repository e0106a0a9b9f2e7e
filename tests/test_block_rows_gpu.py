"""Layer norm of broadcast rows, as ``expand`` makes them and autograd hands
over for a sum over rows, against its definition in 64 bits."""
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


def against_reference(got, x, w, b, dy):
    cols = x.shape[-1]
    flat = {n: None if t is None else t.reshape(-1, cols) if t.dim() > 1 and n not in ("mean", "rstd") else t.reshape(-1)
            for n, t in got.items()}
    for name, (value, bound) in br.layer_norm(x.reshape(-1, cols), w, b, 1e-6, dy.reshape(-1, cols)).items():
        br.check(flat[name], value, bound, name)


# few and many rows, whole vectors and not, short and long: each of the ways to the rows
@pytest.mark.parametrize("rows,cols,dtype", [
    (2, 64, BF), (37, 6144, BF), (2000, 6144, BF), (1300, 12288, FP), (30000, 128, FP), (700, 6144, F32), (2000, 1000, F32),
    (40001, 131, BF), (1301, 6143, FP), (700, 12001, BF), (9999, 515, F32), (640, 5001, F32), (640, 15001, FP)])
@pytest.mark.parametrize("weight", [False, True])
def test_gradient_of_a_sum_over_rows(rows, cols, dtype, weight):
    x, g = rand((rows, cols), dtype, 1, 2.0, 1.0), rand((cols,), dtype, 2)
    w, b = (rand((cols,), F32, 3, 0.3, 1.0), rand((cols,), F32, 4)) if weight else (None, None)
    dy = g.expand(rows, cols)
    y, mean, rstd = gn.layer_norm(x, w, b)
    dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
    against_reference(dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db), x, w, b, dy)
    same = gn.layer_norm_backward(dy.contiguous(), x, mean, rstd, w)
    assert all(p is q or torch.equal(p, q) for p, q in zip(same, (dx, dw, db)))


@pytest.mark.parametrize("docs,tokens,cols,dtype", [(3, 5, 64, BF), (1, 9, 33, F32), (5, 1, 128, FP), (4, 700, 1536, BF), (300, 7, 131, FP)])
def test_three_axes(docs, tokens, cols, dtype):
    x = rand((docs, tokens, cols), dtype, 5, 2.0, 1.0)
    w, b = rand((cols,), F32, 6, 0.3, 1.0), rand((cols,), F32, 7)
    y, mean, rstd = gn.layer_norm(x, w, b)
    for g in (rand((cols,), dtype, 8), rand((tokens, cols), dtype, 9), rand((docs, 1, cols), dtype, 10), rand((1, 1, cols), dtype, 11)):
        dy = g.expand(docs, tokens, cols)
        dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
        against_reference(dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db), x, w, b, dy)
        # x broadcast too: rows that share their input
        xe = rand(g.shape, dtype, 12, 2.0, 1.0).expand(docs, tokens, cols)
        ye, me, re = gn.layer_norm(xe, w, b)
        de = gn.layer_norm_backward(dy, xe, me, re, w)
        against_reference(dict(y=ye, mean=me, rstd=re, dx=de[0], dw=de[1], db=de[2]), xe, w, b, dy)


def test_sum_through_autograd():
    """What autograd hands a layer norm whose output is summed over its rows."""
    x = rand((700, 512), F32, 13, 2.0, 1.0)
    handed = []

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            y, mean, rstd = gn.layer_norm(t.detach())
            ctx.save_for_backward(t, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            handed.append(dy)
            t, mean, rstd = ctx.saved_tensors
            return gn.layer_norm_backward(dy, t.detach(), mean, rstd)[0]

    leaf = x.clone().requires_grad_()
    weights = rand((512,), F32, 14)
    Norm.apply(leaf).sum(0).mul(weights).sum().backward()
    assert handed[0].stride(0) == 0
    value, bound = br.layer_norm(x, None, None, 1e-6, handed[0])["dx"]
    br.check(leaf.grad, value, bound, "dx")


def test_broadcast_outputs_are_refused():
    x = rand((6, 64), BF, 15)
    for out in (rand((1, 64), BF, 16), rand((64,), BF, 16)):
        with pytest.warns(UserWarning):
            assert gn.layer_norm(x, out=out.expand(6, 64)) is None
    y, mean, rstd = gn.layer_norm(x)
    keep = rand((1, 64), BF, 17)
    row = keep.clone()
    with pytest.warns(UserWarning):
        assert gn.layer_norm_backward(x, x, mean, rstd, out=row.expand(6, 64)) is None
    wide = row.expand(6, 64)
    with pytest.warns(UserWarning):                          # nor a broadcast input in place
        assert gn.layer_norm(wide, out=wide) is None
    cube = rand((3, 4, 64), BF, 18)
    with pytest.warns(UserWarning):
        assert gn.layer_norm(cube, out=rand((4, 64), BF, 19).expand(3, 4, 64)) is None
    torch.cuda.synchronize()
    assert torch.equal(row, keep)


@pytest.mark.parametrize("rows,cols", [(9, 256), (1, 128), (3, 64), (17, 255), (5, 1003), (1025, 32)])
def test_gradient_in_place_whose_last_row_overflows(rows, cols):
    """dx written over x, past fp16's range in the last row: the threads that have
    no row beside it bring none of its infinities into the weight's gradient."""
    for n in range(10):
        x, dy = rand((rows, cols), FP, 20 + n, 2.0 ** -12), rand((rows, cols), FP, 40 + n)
        dy[-1, ::2] = 6e4
        w, b = rand((cols,), F32, 3, 0.3, 1.0), rand((cols,), F32, 4)
        y, mean, rstd = gn.layer_norm(x, w, b, eps=1e-12)
        dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w)
        assert torch.isinf(dx[-1]).any() and torch.isfinite(dw).all() and torch.isfinite(db).all()
        onto = x.clone()
        again = gn.layer_norm_backward(dy, onto, mean, rstd, w, out=onto)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
