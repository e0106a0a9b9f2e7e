"""Rows that begin at any element, out of a wider tensor: the elements of the
tensor's first and last blocks are put into shared memory by whichever thread
has the row, and every reader has to find them there."""
import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    gs.lib()
    yield
    gu.assert_clean_device()


# (rows of 131 and 67: batches of 24 and 48, the last row at every place of one; 1003 and 2051: of a few rows)
@pytest.mark.parametrize("cols,start,wide,rows,step", [(131, 5, 140, 15001, 5), (67, 1, 71, 29501, 11), (1003, 3, 1010, 5003, 1),
                                                       (2051, 1, 2053, 2503, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_first_and_last_rows_of_every_batch_length(cols, start, wide, rows, step, dtype):
    gen = torch.Generator().manual_seed(cols)
    most = rows + 12 * step
    x, dy = (torch.randn(most, wide, generator=gen).to(dtype).cuda()[:, start:start + cols] for _ in range(2))
    w, b = torch.randn(cols, generator=gen).cuda(), torch.randn(cols, generator=gen).cuda()
    # the same rows end to end, whose ends lie with the first thread: a row's result does not depend on where it lies
    xc, dyc = x.contiguous(), dy.contiguous()
    y, mean, rstd = gn.layer_norm(xc, w, b)
    dx = gn.layer_norm_backward(dyc, xc, mean, rstd, w)[0]
    for n in range(rows, most, step):
        for lo in (0, 1):
            part = slice(lo, n)
            got, m, r = gn.layer_norm(x[part], w, b)
            assert torch.equal(got, y[part]) and torch.equal(m, mean[part]) and torch.equal(r, rstd[part]), n
            grad = gn.layer_norm_backward(dy[part], x[part], m, r, w)[0]
            assert torch.equal(grad, dx[part]), n
