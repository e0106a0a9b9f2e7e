"""Packed attention with caps of any size: a capped score is as exact as an uncapped one,
however far it is from its cap, for few queries of a document and for many."""
import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from tests import block_ref as br
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    yield
    gu.assert_clean_device()


@pytest.mark.parametrize("cap", [0.01, 0.7, 3.0, 50.0, 1e3, 1e5, 1e9])
@pytest.mark.parametrize("new", [1, 5, 200])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_caps_of_any_size(new, dtype, cap):
    gen = torch.Generator("cuda").manual_seed(new)
    h, hk, dim, lens = 8, 2, 64, [300 + new, 2000]
    cu_q, cu_k = [0, new, 2 * new], [0, lens[0], sum(lens)]
    q, k, v = (torch.randn(s, generator=gen, device="cuda").to(dtype)
               for s in ((2 * new, h, dim), (sum(lens), hk, dim), (sum(lens), hk, dim)))
    ends = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k)]
    out, lse = gn.attention_packed(q, k, v, *ends, causal=True, cap=cap)
    want, plain = br.attention(q, k, v, cu_q, cu_k, causal=True, cap=cap), br.attention(q, k, v, cu_q, cu_k, causal=True)
    # the bounds of uncapped scores, and of the capped ones' tanh 16 roundings of the score
    size = float(q.double().norm(dim=2).amax() * k.double().norm(dim=2).amax()) * dim ** -0.5
    more = 16 * br.U32 * min(size, cap)
    br.check(out, want["out"][0], plain["out"][1] + 2 * (more + br.half_step(dtype)) * v.double().abs().amax(), "out")
    br.check(lse, want["lse"][0], plain["lse"][1] + more + 4 * br.U32 * want["lse"][0].abs(), "lse")
