"""Packed attention's backward pass where its kernels' products take next to no
time (narrow heads, many short tiles), so that the scores of two blocks are
done almost at once, and for head layouts at the ends of the range."""
import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from tests import block_ref as br
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    gs.lib()
    yield
    gu.assert_clean_device()


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dim", [8, 16, 64])
@pytest.mark.parametrize("how", [dict(), dict(causal=True), dict(cap=8.0), dict(bias=True)])
def test_two_blocks_of_scores_in_hand(dim, how):
    """Keys of one to five blocks, call after call beside work on another stream:
    the same bits every time, and those of the formulas."""
    how = dict(how)
    lens = [513, 128, 129, 256, 257, 1, 640]
    cu = [sum(lens[:n]) for n in range(len(lens) + 1)]
    t, h = cu[-1], 6
    if how.pop("bias", False):
        how["slopes"] = 2.0 ** -torch.arange(1, h + 1, device="cuda").float()
    q, k, v, dout = (rand((t, h, dim), BF, s, 1.5) for s in (1, 2, 3, 4))
    ends = i32(cu)
    out, lse = gn.attention_packed(q, k, v, ends, ends, **how)
    first = gn.attention_packed_backward(dout, q, k, v, out, lse, ends, ends, **how)
    want = br.attention(q, k, v, cu, cu, dout=dout, **how)
    for name, got in zip(("dq", "dk", "dv"), first):
        br.check(got, *want[name], name)
    side = torch.cuda.Stream()
    other = torch.randn(2048, 2048, device="cuda")
    for n in range(60):
        if n % 4 == 0:
            with torch.cuda.stream(side):
                other = other @ other * 2.0 ** -11
        again = gn.attention_packed_backward(dout, q, k, v, out, lse, ends, ends, **how)
        assert all(torch.equal(a, b) for a, b in zip(again, first)), n
    side.synchronize()
