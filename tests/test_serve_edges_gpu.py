"""Attention over the paged cache where products and sums leave the ordinary range: zero
queries and keys, pages that there are not, scales of 0."""
import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from tests import block_ref as br
from tests import gpu_util as gu
from tests import serve_ref as sr

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    yield
    gu.assert_clean_device()


def rand(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype).cuda()


def attend(q, cache, begins, what, **how):
    cu = torch.tensor(begins, dtype=torch.int32, device="cuda")
    out, lse = gn.attention_cached(q, *cache.args(), cu, **how)
    want = sr.attention(q, cache, begins, **how)
    br.check(out, *want["out"], f"out {what}")
    br.check(lse, *want["lse"], f"lse {what}")
    return out, lse


HOW = [dict(), dict(cap=5.0), dict(causal=False)]


@pytest.mark.parametrize("page", [8, 24, 32, 64])
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new", [1, 5, 70, 300])
def test_zero_queries_over_zero_keys(new, dtype, how, page):
    """What a padded prompt holds: the append gives zero keys the least scale."""
    cache = sr.Cache([new + 17, new], page, 2, 64, seed=1)
    zero = torch.zeros(2 * new, 2, 64, dtype=dtype, device="cuda")
    v = rand(zero.shape, dtype, 2)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    assert gn.cache_append(zero, v, *cache.args(), cu) is True
    q = torch.zeros(2 * new, 8, 64, dtype=dtype, device="cuda")
    _, lse = attend(q, cache, [0, new, 2 * new], f"{new} zero queries", **how)
    assert lse.isfinite().all()
    q[::3] = rand(q[::3].shape, dtype, 3)                 # some of them are not zero
    attend(q, cache, [0, new, 2 * new], f"{new} queries over zero keys", **how)


@pytest.mark.parametrize("page", [8, 24, 32, 64])
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new", [1, 5, 70, 300])
def test_pages_that_there_are_not_and_scales_of_zero(new, dtype, how, page):
    """They read as zeros, under the diagonal too."""
    lens = [new + 200, new + 3]
    q = rand((2 * new, 8, 64), dtype, 3)
    for gone in (-1, 10 ** 6):
        cache = sr.Cache(lens, page, 2, 64, seed=2)
        for s in range(2):
            for place in (lens[s] - 1, 60):
                cache.table_host[s][min(place, lens[s] - 1) // page] = gone
        cache.table = torch.tensor(cache.table_host, dtype=torch.int32, device="cuda")
        out, lse = attend(q, cache, [0, new, 2 * new], f"{new} without pages", **how)
        assert out.isfinite().all() and lse.isfinite().all()
    cache = sr.Cache(lens, page, 2, 64, seed=2)
    for s in range(2):
        cache.k_scales[cache.table_host[s][(lens[s] - 1) // page]] = 0.0
        cache.k_scales[cache.table_host[s][0], 1] = 0.0
    out, lse = attend(q, cache, [0, new, 2 * new], f"{new} with scales of 0", **how)
    assert out.isfinite().all() and lse.isfinite().all()


def test_scales_far_apart_in_one_call():
    """Key scales from the least on, queries from the least half number on."""
    cache = sr.Cache([500], 32, 1, 64, seed=3)
    places = cache.table_host[0]
    for n, at in enumerate(places):
        cache.k_scales[at] = 2.0 ** (-100 + 7 * n) if 2.0 ** (-100 + 7 * n) < 1e-2 else 2.0 ** -8
    for new in (2, 130):
        q = rand((new, 4, 64), BF, 4)
        q *= torch.exp2(-(4.0 * torch.arange(new, device="cuda") % 128))[:, None, None].to(BF)
        attend(q, cache, [0, new], f"{new} queries of all sizes")


@pytest.mark.parametrize("cap", [1e-38, 1e-9, 0.01, 0.7, 3.0, 50.0, 1e3, 1e5, 1e9, 1e20, 9e37])
@pytest.mark.parametrize("new", [1, 5, 70])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_caps_of_any_size(new, dtype, cap):
    """A capped score is as exact as an uncapped one, however far it is from its cap."""
    cache = sr.Cache([new + 300, new], 32, 2, 64, seed=5)
    begins = [0, new, 2 * new]
    q = rand((2 * new, 8, 64), dtype, 6)
    cu = torch.tensor(begins, dtype=torch.int32, device="cuda")
    out, lse = gn.attention_cached(q, *cache.args(), cu, cap=cap)
    want, plain = sr.attention(q, cache, begins, cap=cap), sr.attention(q, cache, begins)
    # the bounds of uncapped scores, and of the capped ones' tanh 16 roundings of the score
    size = max(float((cache.values("k", s).norm(dim=2).amax() * q.double().norm(dim=2).amax() / 8)) for s in range(2))
    more = 16 * br.U32 * min(size, cap)
    v = max(float(cache.values("v", s).abs().amax()) for s in range(2))
    br.check(out, want["out"][0], plain["out"][1] + 2 * (more + br.half_step(dtype)) * v, "out")
    br.check(lse, want["lse"][0], plain["lse"][1] + more + 4 * br.U32 * want["lse"][0].abs(), "lse")
