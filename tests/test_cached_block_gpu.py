"""The example block (examples/cached_block.py) that runs the operators of serving
together, against the same step in 64 bits over what its cache holds."""
import importlib.util
import os

import pytest
import torch

from channels_last_groupnorm_gb300 import build as gnbuild
from tests import block_ref as br
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    spec = importlib.util.spec_from_file_location("cached_block", os.path.join(ROOT, "examples", "cached_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    gu.assert_clean_device()


def plain(ex, block, cache, x, residual, positions, new):
    """(update, total, keys and values of the new tokens), attention over what the cache holds."""
    h, hk, d = block.heads, block.kv_heads, block.dim
    total = (x.float() + residual.float()).bfloat16().double()
    y = total / torch.sqrt((total * total).mean(1, keepdim=True) + ex.EPS) * block.norm.double()
    qkv = (y @ block.w_qkv.double()).view(-1, h + 2 * hk, d)
    q, _ = br.rope(qkv[:, :h], positions, ex.AXES, ex.THETA, True, False)
    k, _ = br.rope(qkv[:, h:h + hk], positions, ex.AXES, ex.THETA, True, False)
    outs, at = [], 0
    for s, n in enumerate(new):
        length, pages = cache.held[s], torch.tensor(cache.rows[s], device=x.device)
        kv = [(p[pages].double() * c[pages].double()[:, None, :, None]).flatten(0, 1)[:length].repeat_interleave(h // hk, 1)
              for p, c in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales))] if length else None
        if n:
            scores = torch.einsum("ihd,jhd->hij", q[at:at + n], kv[0]) / d ** 0.5
            late = torch.arange(length, device=x.device) > torch.arange(length - n, length, device=x.device)[:, None]
            outs.append(torch.einsum("hij,jhd->ihd", scores.masked_fill(late, -torch.inf).softmax(-1), kv[1]))
        at += n
    return torch.cat(outs).flatten(1) @ block.w_o.double(), total, k, qkv[:, h + hk:]


def test_cached_block_in_chunks_and_single_tokens(example):
    block = example.CachedBlock(channels=256, heads=4, kv_heads=2, dim=128, seed=3)
    cache = example.PagedCache(sequences=3, pages=24, kv_heads=2, page_size=32)
    gen = torch.Generator().manual_seed(1)
    for new in ([100, 33, 0], [1, 70, 2], [1, 1, 1], [1, 1, 1], [0, 40, 300], [1, 1, 1]):
        cu = cache.grow(new)
        x, residual = (torch.randn(2, sum(new), 256, generator=gen) * 1.5).bfloat16().cuda()
        positions = example.places(cache.held, new)
        update, total = block.step(x, residual, positions, cache, cu)
        want, stream, k, v = plain(example, block, cache, x, residual, positions, new)
        assert torch.equal(total.double(), stream)
        # Three roundings to bf16 ahead of the scores (2^-9 each of a query's norm, scores of up to
        # four deviations), two behind them: under 2^-4 of the result's norm.
        assert (update.double() - want).norm() < 2.0 ** -4 * want.norm(), new
        # the new tokens are where they belong, within e4m3's half step and the product's roundings
        at = 0
        for s, n in enumerate(new):
            for i in range(n):
                place = cache.held[s] - n + i
                page, slot = cache.rows[s][place // 32], place % 32
                for pool, scales, wanted in ((cache.k_pages, cache.k_scales, k), (cache.v_pages, cache.v_scales, v)):
                    got = pool[page, slot].double() * scales[page].double()[:, None]
                    close = (2.0 ** -4 + 2.0 ** -7) * wanted[at + i].abs() + 2.0 ** -6 + 2.0 ** -10 * scales[page].double()[:, None]
                    assert ((got - wanted[at + i]).abs() <= close).all(), (s, place)
            at += n
