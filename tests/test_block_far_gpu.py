"""The transformer-block operators on tensors of more than 2^31 elements: what
lies past that is what the same rows and tokens give by themselves."""
import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from tests import block_ref as br
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    gnbuild.build()
    gs.lib()
    yield
    torch.cuda.empty_cache()
    gu.assert_clean_device()


def far(shape):
    """A tensor whose first and last 4096 rows or tokens hold normal values."""
    gen = torch.Generator().manual_seed(len(shape) + shape[-1])
    t = torch.zeros(shape, dtype=BF, device="cuda")
    for part in (t[:4096], t[-4096:]):
        part.copy_(torch.randn(part.shape, generator=gen).to(BF))
    return t


@pytest.mark.parametrize("rows,cols", [(530000, 4096), (530500, 4095), (180000, 12288), (17200000, 128)])
def test_layer_norm(rows, cols):
    assert rows * cols > 1 << 31
    x, dy, w = far((rows, cols)), far((rows, cols)), torch.ones(cols, device="cuda")
    y, mean, rstd = gn.layer_norm(x, w)
    dx, dw, db = gn.layer_norm_backward(dy, x, mean, rstd, w, out=dy.clone())
    for part in (slice(0, 4096), slice(rows - 4096, rows)):
        want = br.layer_norm(x[part], w, None, 1e-6, dy[part])
        for name, got in dict(y=y, mean=mean, rstd=rstd, dx=dx).items():
            br.check(got[part], *want[name], name)
    ends = torch.cat([dy[:4096], dy[-4096:]]), torch.cat([x[:4096], x[-4096:]])
    want = br.layer_norm(ends[1], w, None, 1e-6, ends[0])     # (the rows between have dy 0)
    br.check(dw, *want["dw"], "dw")
    br.check(db, *want["db"], "db")


def test_rotation():
    q = far((2200000, 8, 128))
    assert q.numel() > 1 << 31
    pos = torch.arange(2 * q.shape[0], device="cuda", dtype=torch.int32).view(-1, 2)
    got, _ = gn.rope_nd(q, None, pos, [64, 64])
    for part in (slice(0, 4096), slice(q.shape[0] - 4096, q.shape[0])):
        br.check(got[part], *br.rope(q[part], pos[part], [64, 64], 1e4, True, False), "rope")


@pytest.mark.parametrize("lens", [[1, 1], [300, 700]])
def test_attention_of_a_document_behind_a_long_cache(lens):
    """Documents in the first and the last keys of a cache, none in what lies between."""
    k, v = far((2200000, 8, 128)), far((2200000, 8, 128))
    assert k.numel() > 1 << 31
    tk, tq = k.shape[0], sum(lens)
    gen = torch.Generator().manual_seed(3)
    q, dout = (torch.randn(tq, 16, 128, generator=gen).to(BF).cuda() for _ in range(2))
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    cu_q, cu_k = i32([0, lens[0], lens[0], tq]), i32([0, 1000, tk - 2000, tk])
    out, lse = gn.attention_packed(q, k, v, cu_q, cu_k, causal=True)
    dq, dk, dv = gn.attention_packed_backward(dout, q, k, v, out, lse, cu_q, cu_k, causal=True)
    for qs, ks in ((slice(0, lens[0]), slice(0, 1000)), (slice(lens[0], tq), slice(tk - 2000, tk))):
        n, m = qs.stop - qs.start, ks.stop - ks.start
        want = br.attention(q[qs], k[ks], v[ks], [0, n], [0, m], causal=True, dout=dout[qs])
        for name, got in dict(out=out[qs], lse=lse[:, qs], dq=dq[qs], dk=dk[ks], dv=dv[ks]).items():
            br.check(got, *want[name], name)
    assert not dk[1000:tk - 2000].any() and not dv[1000:tk - 2000].any()
