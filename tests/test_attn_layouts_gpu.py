"""Head layouts of packed attention at the ends of the range: more query heads
per key / value head than a tile has rows, odd numbers of them, and few rows
of every count."""
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


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def check(q_lens, k_lens, h, hk, dim, dtype, backward, **how):
    cu_q, cu_k = ([sum(n[:i]) for i in range(len(n) + 1)] for n in (q_lens, k_lens))
    ends = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k)]
    q, k, v = (rand((n, m, dim), dtype, s, 1.3) for n, m, s in ((cu_q[-1], h, 1), (cu_k[-1], hk, 2), (cu_k[-1], hk, 3)))
    dout = rand(q.shape, dtype, 4) if backward else None
    out, lse = gn.attention_packed(q, k, v, *ends, **how)
    got = dict(out=out, lse=lse)
    if backward:
        got |= dict(zip(("dq", "dk", "dv"), gn.attention_packed_backward(dout, q, k, v, out, lse, *ends, **how)))
    for name, (value, bound) in br.attention(q, k, v, cu_q, cu_k, dout=dout, **how).items():
        br.check(got[name], value, bound, name)


# 129 and 200 heads to one key head: two tiles of heads for each token, the last one partly past the group
@pytest.mark.parametrize("h,hk", [(128, 1), (129, 1), (200, 1), (260, 2), (300, 2)])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, FP)])
def test_more_heads_to_a_key_head_than_a_tile_has_rows(h, hk, dim, dtype):
    for how in (dict(causal=True), dict(cap=15.0, slopes=torch.linspace(0.01, 0.2, h, device="cuda"))):
        check([1, 1, 1], [900, 1, 333], h, hk, dim, dtype, False, **how)
        check([2, 1, 3], [300, 128, 3], h, hk, dim, dtype, False, **how)


@pytest.mark.parametrize("h,hk", [(7, 1), (14, 2), (5, 1), (9, 3), (15, 3), (21, 1), (49, 7), (11, 1)])
def test_odd_numbers_of_heads_to_a_key_head(h, hk):
    for how in (dict(), dict(cap=15.0, causal=True)):
        check([130, 1, 261], [130, 1, 261], h, hk, 64, BF, True, **how)
        check([130, 1, 61], [130, 1, 61], h, hk, 128, FP, True, **how)


@pytest.mark.parametrize("h,hk,new", [(3, 1, 1), (5, 1, 3), (15, 1, 1), (17, 1, 1), (31, 1, 1), (33, 1, 1), (11, 1, 3), (57, 1, 1),
                                      (57, 1, 2), (63, 1, 2), (100, 1, 1)])
@pytest.mark.parametrize("dim", [40, 128])
def test_every_count_of_few_rows(h, hk, new, dim):
    for how in (dict(causal=True), dict(cap=20.0)):
        check([new] * 3, [700, new, 129], h, hk, dim, BF, False, **how)


def test_cache_with_room_behind_each_document():
    """Room is told by documents without queries; whatever it holds changes nothing."""
    lens, room = [700, 1, 129, 333, 50], [68, 127, 383, 179, 14]
    q = rand((5, 16, 128), BF, 1)
    k, v = (rand((sum(lens), 4, 128), BF, s) for s in (2, 3))
    ends = lambda e: torch.tensor(e, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [sum(lens[:n]) for n in range(6)]
    want = br.attention(q, k, v, list(range(6)), cu, causal=True)
    for fill in (0.0, float("nan")):
        wide_k, wide_v = (torch.full((sum(lens) + sum(room), 4, 128), fill, dtype=BF, device="cuda") for _ in range(2))
        cu_q, cu_k, at = [0], [0], 0
        for n, (length, free) in enumerate(zip(lens, room)):
            wide_k[at:at + length], wide_v[at:at + length] = k[cu[n]:cu[n + 1]], v[cu[n]:cu[n + 1]]
            at += length + free
            cu_q += [n + 1, n + 1]
            cu_k += [at - free, at]
        out, lse = gn.attention_packed(q, wide_k, wide_v, ends(cu_q), ends(cu_k), causal=True)
        br.check(out, *want["out"], "out")
        br.check(lse, *want["lse"], "lse")


@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("q_lens,k_lens,h,hk,dim", [([200, 7], [200, 300], 2, 2, 64), ([1, 1], [300, 5], 8, 2, 128), ([3, 2], [300, 70], 40, 2, 64)])
def test_scales_that_are_not_positive(q_lens, k_lens, h, hk, dim, scale):
    for how in (dict(), dict(cap=3.0), dict(slopes=torch.full((h,), 0.05, device="cuda")), dict(causal=True)):
        check(q_lens, k_lens, h, hk, dim, BF, True, scale=scale, **how)


def test_norm_and_rotation_on_another_stream():
    """The work lands on the stream that was named, and its inputs may be let go at once."""
    x, w, b = rand((3001, 1536), BF, 1, 2.0), rand((1536,), F32, 2), rand((1536,), F32, 3)
    dy = rand(x.shape, BF, 4)
    q, k = rand((500, 6, 128), BF, 5), rand((500, 2, 128), BF, 6)
    pos = torch.arange(1000, device="cuda", dtype=torch.int32).view(500, 2)
    y, mean, rstd = gn.layer_norm(x, w, b)
    grads = gn.layer_norm_backward(dy, x, mean, rstd, w)
    turned = gn.rope_nd(q, k, pos, [64, 64])
    side = torch.cuda.Stream()
    for _ in range(20):
        inputs = [t.clone() for t in (x, w, b, dy, q, k, pos)]
        side.wait_stream(torch.cuda.current_stream())
        xc, wc, bc, dyc, qc, kc, pc = inputs
        y2, m2, r2 = gn.layer_norm(xc, wc, bc, stream=side)
        g2 = gn.layer_norm_backward(dyc, xc, m2, r2, wc, stream=side)
        t2 = gn.rope_nd(qc, kc, pc, [64, 64], stream=side)
        del inputs, xc, wc, bc, dyc, qc, kc, pc
        torch.empty(3001, 1536, device="cuda", dtype=BF).fill_(7.0)
    side.synchronize()
    assert torch.equal(y2, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)
    assert all(torch.equal(p, s) for p, s in zip(g2 + t2, grads + turned))


def test_norm_and_rotation_in_a_graph():
    """Forward and backward captured together, replayed on new inputs."""
    x, w, b = rand((2003, 1000), BF, 1, 2.0), rand((1000,), F32, 2), rand((1000,), F32, 3)
    dy = rand(x.shape, BF, 4)
    q, k = rand((500, 6, 128), BF, 5), rand((500, 2, 128), BF, 6)
    pos = torch.arange(1000, device="cuda", dtype=torch.int32).view(500, 2)

    def run():
        y, mean, rstd = gn.layer_norm(x, w, b)
        return (y, mean, rstd, *gn.layer_norm_backward(dy, x, mean, rstd, w), *gn.rope_nd(q, k, pos, [64, 64]))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for seed in (7, 8):
        x.copy_(rand(x.shape, BF, seed))
        q.copy_(rand(q.shape, BF, seed))
        pos.add_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(captured, run()))
