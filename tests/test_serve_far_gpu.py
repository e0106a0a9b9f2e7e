"""RMS norm and the paged cache on tensors of more than 2^31 elements and pools of
more than 2^32 bytes, on other streams at once, and in captured calls."""
import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from tests import block_ref as br
from tests import gpu_util as gu
from tests import serve_ref as sr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    yield
    gu.assert_clean_device()


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def test_rms_norm_of_more_than_2_31_elements():
    rows, cols = 350_003, 6144
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 1, 174_001, 349_525, 349_526, rows - 1], device="cuda")
    x[some] = rand((6, cols), 1, 2.0)
    residual = torch.zeros_like(x)
    residual[some] = rand((6, cols), 2, 2.0)
    w = rand((cols,), 3, 0.2, torch.float32) + 1.0
    y, scales, total, rstd = gn.rms_norm(x, w, residual=residual, total_out=residual, quantize=True)
    t = total[some].double()
    value = t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6) * w.double()
    got = y[some].double() * scales[some].double()[:, None]
    br.check(got, value, (2.0 ** -4 + 2.0 ** -15) * value.abs() + 2.0 ** -10 * value.abs().amax(1, keepdim=True) / 448, "rows")
    assert int((scales != 0).sum()) == 6 and total is residual
    del y, scales
    dy = x                      # the gradient of the same few rows
    dx, dw = gn.rms_norm_backward(dy, total, rstd, w)
    part = sr.rms_norm(total[some], w, 1e-6, dy=dy[some])
    br.check(dx[some], *part["dx"], "dx")
    br.check(dw, part["dw"][0], part["dw"][1] + rows * 2.0 ** -24 * part["dw"][0].abs(), "dw")


def test_cache_pages_past_2_32_bytes():
    """A few sequences whose pages lie at the far end of pools of 5 GB each."""
    pages, page, hk, dim, h = 20_000, 256, 8, 128, 16
    pools = [torch.zeros(pages, hk, page, dim, dtype=torch.uint8, device="cuda").view(sr.E4M3).transpose(1, 2) for _ in range(2)]
    scales = [torch.zeros(pages, hk, device="cuda") for _ in range(2)]
    table = torch.tensor([[19_999, 0, 16_385], [16_384, 19_998, 1]], dtype=torch.int32, device="cuda")
    lens = [700, 513]
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 700, 1213], dtype=torch.int32, device="cuda")
    k, v = rand((1213, hk, dim), 1, 1.5), rand((1213, hk, dim), 2)
    args = (*pools, *scales, table, lengths)
    assert gn.cache_append(k, v, *args, cu) is True
    cache = sr.Cache.__new__(sr.Cache)
    cache.lens, cache.page, cache.table_host, cache.table = lens, page, table.tolist(), table
    for name, pool, scale in zip("kv", pools, scales):
        setattr(cache, name + "_bytes", pool.view(torch.uint8))
        setattr(cache, name + "_scales", scale)
    for name, x in (("k", k), ("v", v)):
        for s, (a, b) in enumerate(((0, 700), (700, 1213))):
            got = cache.values(name, s)
            step = 2.0 ** -4 * x[a:b].double().abs() + 2.0 ** -10 * scales["kv".index(name)].double().amax()
            br.check(got, x[a:b].double(), step, f"{name} of {s}")
    for new in ([1, 1], [70, 300]):
        q = rand((sum(new), h, dim), 5, 1.5)
        ends = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        out, lse = gn.attention_cached(q, *args, ends)
        want = sr.attention(q, cache, [0, new[0], sum(new)])
        br.check(out, *want["out"], f"out {new}")
        br.check(lse, *want["lse"], f"lse {new}")


def test_two_calls_at_once_on_streams_of_their_own():
    caches = [sr.Cache([900, 4000], 64, 2, 128, seed=s) for s in (1, 2)]
    queries = [[rand((n, 8, 128), s + n, 1.5) for n in (2, 600)] for s in (3, 4)]
    alone = [[gn.attention_cached(q, *c.args()) for q in qs] for c, qs in zip(caches, queries)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[gn.attention_cached(q, *c.args(), stream=s) for q in qs] for s, c, qs in zip(streams, caches, queries)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_a_captured_step_replayed_on_growing_caches():
    """Norm, append and attention in one graph: lengths grow between replays."""
    cache, eager = (sr.Cache([5, 64, 31], 32, 2, 64, seed=1, spare=8, width=4) for _ in range(2))
    for c in (cache, eager):
        free = [p for p in range(c.k_pages.shape[0]) if p not in {r for row in c.table_host for r in row}]
        for row in range(3):
            for i in range(4):
                if c.table_host[row][i] < 0:
                    c.table_host[row][i] = free.pop()
        c.table = torch.tensor(c.table_host, dtype=torch.int32, device="cuda")
    x, r, qkv, pos = rand((3, 512), 2), rand((3, 512), 3), rand((3, 8, 64), 4), torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    w = rand((512,), 5)

    def step(c):
        y, scales, total, _ = gn.rms_norm(x, w, residual=r, quantize=True)
        q = gn.cache_append(qkv[:, 4:6], qkv[:, 6:], *c.args(), q=qkv[:, :4], positions=pos, axes_dim=(64,))
        return y, scales, total, *gn.attention_cached(q, *c.args())

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(cache)
    for n in range(40):
        for c in (cache, eager):
            c.lengths += 1
        pos.copy_(cache.lengths[:, None] - 1)
        qkv.copy_(rand(qkv.shape, 10 + n, 1.0 + n / 8))
        x.copy_(rand(x.shape, 90 + n))
        graph.replay()
        for a, b in zip(outs, step(eager)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
    for name in "kv":
        assert torch.equal(cache.pages(name), eager.pages(name))
        assert torch.equal(cache.scales(name).nan_to_num(-1), eager.scales(name).nan_to_num(-1))
