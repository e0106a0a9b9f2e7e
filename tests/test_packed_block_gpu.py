"""The example block (examples/packed_image_block.py) that runs the
transformer-block operators together, against the same block from elementary
torch operations in 64 bits and its automatic gradients."""
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
    spec = importlib.util.spec_from_file_location("packed_image_block",
                                                  os.path.join(ROOT, "examples", "packed_image_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    gu.assert_clean_device()


def plain(ex, block, w, x, positions, ends):
    """The block in 64 bits, one document and head after the other."""
    def norm(t, weight=None):
        c = t - t.mean(-1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + ex.EPS)
        return y if weight is None else y * weight

    def turn(t):
        rate = torch.cat([ex.THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=t.device) / d) for d in ex.AXES])
        axis = torch.repeat_interleave(torch.arange(4, device=t.device), 16)
        angle = (positions.double()[:, axis] * rate)[:, None]
        a, b = t[..., 0::2], t[..., 1::2]
        return torch.stack([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).flatten(-2)

    h, hk, d = block.heads, block.kv_heads, block.dim
    qkv = (norm(x) @ w["w_qkv"]).view(x.shape[0], h + 2 * hk, d)
    q, k, v = turn(norm(qkv[:, :h], w["q_norm"])), turn(norm(qkv[:, h:h + hk], w["k_norm"])), qkv[:, h + hk:]
    e = ends.tolist()
    outs = []
    for lo, hi in zip(e, e[1:]):
        s = torch.einsum("ihd,jhd->hij", q[lo:hi], k[lo:hi].repeat_interleave(h // hk, 1)) / d ** 0.5
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), v[lo:hi].repeat_interleave(h // hk, 1)))
    return x + w["gate"] * (torch.cat(outs).flatten(1) @ w["w_o"])


def test_block_matches_plain_block_and_its_gradients(example):
    block = example.PackedBlock(channels=256, heads=4, kv_heads=2, seed=3)
    ends, positions = example.packed_images([200, 70, 131], [40, 6, 31])
    x = torch.randn(401, 256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dz = torch.randn(401, 256, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    z, kept = block.forward(x, positions, ends)
    grads = block.backward(dz, kept)
    w = {n: getattr(block, n).double().requires_grad_() for n in ("w_qkv", "w_o", "q_norm", "k_norm", "gate")}
    xd = x.double().requires_grad_()
    want = plain(example, block, w, xd, positions, ends)
    want.backward(dz.double())
    # a value passes at most 16 roundings to bf16 on its way (forward: norm, projection,
    # head norm, turn, weights, output, projection, update; as many back), each half a step
    # relative to values of its own size, as independent as rounding is: 2-norms within
    # sqrt(16) of them, and twice that for the norms' and softmax' own conditioning
    bound = 2 * 16 ** 0.5 * br.half_step(torch.bfloat16)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())
    assert off(z, want.detach()) < bound
    assert off(grads["x"], xd.grad) < bound
    for n, g in grads.items():
        if n != "x":
            assert off(g, w[n].grad) < bound, (n, off(g, w[n].grad))


def test_single_tokens_give_what_the_whole_sequence_gives(example):
    block = example.PackedBlock(channels=256, heads=8, kv_heads=2, seed=4)
    ends, positions = example.packed_images([333, 1, 129, 64], [33, 1, 0, 64])
    x = torch.randn(527, 256, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    z, kept = block.forward(x, positions, ends)
    caches = [kept[2].clone(), kept[3].clone().contiguous()]
    last = ends[1:].long() - 1
    for c in caches:
        c[last] = 7.0                                        # the new tokens' own are written by the call
    new = block.decode(x[last], positions[last], caches[0], caches[1], ends)
    # the same numbers summed in another order, rounded to bf16 four times after that
    err = (new.double() - z[last].double()).norm() / z[last].double().norm()
    assert float(err) < 4 * br.half_step(torch.bfloat16)
