"""Attention over the paged cache at the sizes of long prompts and large batches, where every
CTA has many tiles, against its definition in 64 bits."""
import math

import pytest
import torch

import channels_last_groupnorm_gb300 as gn
from channels_last_groupnorm_gb300 import build as gnbuild
from tests import block_ref as br
from tests import gpu_util as gu
from tests import serve_ref as sr

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
U32 = br.U32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gnbuild.build()
    yield
    gu.assert_clean_device()


class Even:
    """A cache of sequences of equally many tokens, made on the GPU."""

    def __init__(self, count, length, hk, dim, page=64, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        width = (length + page - 1) // page
        self.length, self.page = length, page
        self.table = torch.randperm(count * width, generator=gen, device="cuda").to(torch.int32).view(count, width)
        self.lengths = torch.full((count,), length, dtype=torch.int32, device="cuda")
        for name in "kv":
            x = torch.randn(count * width, hk, page, dim, generator=gen, device="cuda")
            scale = torch.exp2(torch.randint(-9, -5, (count * width, hk), generator=gen, device="cuda").float())
            setattr(self, name + "_pages", (x * 128.0).clamp(-448.0, 448.0).to(sr.E4M3).transpose(1, 2))
            setattr(self, name + "_scales", scale)

    def args(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales, self.table, self.lengths

    def values(self, name, head):
        """[sequences, length, dim] in 64 bits."""
        pages, scales = getattr(self, name + "_pages")[:, :, head], getattr(self, name + "_scales")[:, head]
        x = pages.float().double() * scales.double()[:, None, None]
        return x[self.table.long()].flatten(1, 2)[:, :self.length]


def check(q, cache, got, floor, what, scale=None):
    """Causal attention of equally many new tokens for each sequence.  The bound is that of
    serve_ref.attention, but for the weights' floor: `floor` of the row's largest for each key."""
    tokens, h, dim = q.shape
    count, hk = cache.table.shape[0], cache.k_scales.shape[1]
    new = tokens // count
    scale = dim ** -0.5 if scale is None else scale
    u, low = br.half_step(q.dtype), br.least(q.dtype)
    j, place = torch.arange(cache.length, device="cuda"), torch.arange(cache.length - new, cache.length, device="cuda")
    seen = j <= place[:, None]
    for head in range(h):
        k, v = (cache.values(n, head * hk // h) for n in "kv")
        qh = q.view(count, new, h, dim)[:, :, head].double()
        t = qh @ k.transpose(1, 2) * scale
        size = qh.abs() @ k.abs().transpose(1, 2) * abs(scale)
        worst = (U32 * ((dim + 4) * size + 4 * t.abs() + 4)).masked_fill_(~seen, 0.0).amax(2, keepdim=True)
        del size
        t.masked_fill_(~seen, -math.inf)
        lse = torch.logsumexp(t, 2, keepdim=True)
        top = t.amax(2, keepdim=True)
        p = t.sub_(lse).exp_()
        rel = 2 * worst + 2.0 ** -20 + cache.length * U32 / 64
        drop = 2.0 ** -17 * qh.abs().amax(2, keepdim=True) * k.abs().sum(2).amax(1)[:, None, None] * abs(scale)
        out, absout = p @ v, p @ v.abs()
        del p
        least = floor * torch.exp(top - lse)
        off = low + u * out.abs() + (u + rel) * absout + (low + least) * v.abs().sum(1, keepdim=True) + 2 * drop * absout
        br.check(got[0].view(count, new, h, dim)[:, :, head], out, off, f"out of head {head}, {what}")
        br.check(got[1][head].view(count, new), lse[..., 0], (rel + 4 * U32 * lse.abs() + drop)[..., 0], f"lse of head {head}, {what}")


@pytest.mark.parametrize("count,length,new,h,hk,dtype", [
    (296, 700, 1, 32, 32, BF), (1180, 640, 1, 32, 8, BF), (1180, 1000, 1, 32, 8, FP),        # 32 tiles of single tokens a CTA
    (1, 12288, 12288, 64, 2, BF), (1, 10000, 10000, 32, 8, FP), (290, 2000, 64, 32, 8, BF),  # 16 tiles of many tokens a CTA
    (8, 2048, 2048, 32, 8, FP), (64, 3000, 1, 32, 32, BF), (400, 1500, 3, 16, 4, FP)])
def test_every_row_of_large_calls_is_written(count, length, new, h, hk, dtype):
    """Calls in which CTAs begin a tile that others go on with as the last of a full list."""
    dim = 16
    cache = Even(count, length, hk, dim, seed=count)
    q = torch.randn(count * new, h, dim, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    outs = []
    for fill in (math.nan, 7.0):
        out = torch.full_like(q, fill)
        other = torch.full((h, count * new), fill, device="cuda")      # (where the next lse will probably lie)
        del other
        outs.append(gn.attention_cached(q, *cache.args(), out=out))
    (a, a_lse), (b, b_lse) = outs
    assert not a.isnan().any() and not a_lse.isnan().any()
    assert torch.equal(a, b) and torch.equal(a_lse, b_lse)
    check(q, cache, outs[0], 2.0 ** -32, f"{count} x {new} tokens")


@pytest.mark.parametrize("new,keys,h", [(1, 2 ** 24, 1), (3, 2 ** 24, 2), (70, 2 ** 22, 1), (300, 2 ** 21, 4)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_zero_values_of_very_long_sequences(new, keys, h, dtype):
    """Values of the least scale leave the sum of the weights as 2^100 of each.  A page is
    all of the cache: every query sees it keys / 256 times over."""
    gen = torch.Generator("cuda").manual_seed(new)
    k_pages = torch.randn(1, 256, 1, 16, generator=gen, device="cuda").mul(64.0).to(sr.E4M3)
    k_scales, v_scales = torch.full((1, 1), 2.0 ** -8, device="cuda"), torch.full((1, 1), 2.0 ** -100, device="cuda")
    table = torch.zeros(1, keys // 256, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([keys], dtype=torch.int32, device="cuda")
    q = torch.randn(new, h, 16, generator=gen, device="cuda").to(dtype)
    k = k_pages[0, :, 0].float().double() * 2.0 ** -8
    t = torch.einsum("nhd,kd->hnk", q.double(), k) / 4
    lse = torch.logsumexp(t, 2) + math.log(keys // 256)
    # a score's error, and a thread's sum of one key of each of its CTA's blocks (under 2^10 of them)
    size = torch.einsum("nhd,kd->hnk", q.double().abs(), k.abs()) / 4
    drop = 2.0 ** -17 * q.double().abs().amax(2).T * k.abs().sum(1).amax() / 4
    off = drop + U32 * (20 * size.amax(2) + 4 * t.abs().amax(2) + 4) + 2.0 ** -14 + 4 * U32 * lse.abs()
    for values in (0.0, 3.0):
        v_pages = torch.full((1, 256, 1, 16), values, device="cuda").to(sr.E4M3)
        out, got = gn.attention_cached(q, k_pages, v_pages, k_scales, v_scales, table, lengths, causal=False)
        br.check(got, lse, off, "lse")
        want = torch.full(out.shape, values * 2.0 ** -100, dtype=torch.float64, device="cuda")
        if dtype == FP:
            want *= 0                                          # (under half of the least half number)
        br.check(out, want, (br.half_step(dtype) + 2.0 ** -8) * want.abs(), "out")


@pytest.mark.parametrize("count,length,new,h,hk", [(40, 32768, 1, 8, 8), (1, 131072, 3, 16, 8), (2, 32768, 70, 4, 2)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("above", [9, 12, 13, 14, 16])
@pytest.mark.parametrize("even", [False, True])
def test_one_key_far_above_a_long_context(count, length, new, h, hk, dtype, above, even):
    """A key with most of the weight and hardly a value: what comes out is the sum of many
    small weights, which may be off by a rounding of each, and no more.  (even: all alike)"""
    dim = 64
    cache = Even(count, length, hk, dim, seed=above)
    k, v = (getattr(cache, n + "_pages").transpose(1, 2) for n in "kv")           # [pages, head, slot, channel]
    for name, pages, scale in (("k", k, 2.0 ** -4), ("v", v, 2.0 ** -7)):
        getattr(cache, name + "_scales").fill_(scale)
    if even:
        k.view(torch.uint8).zero_()
    else:
        k.copy_((k.float() / 8).to(sr.E4M3))                                        # deviation 1
    # channel 0 is the far key's own; one of it in every sequence
    k.view(torch.uint8)[..., 0] = 0
    at = cache.table[:, cache.table.shape[1] // 2].long()
    far = torch.zeros(dim, device="cuda")
    far[0] = above * 16.0
    k.view(torch.uint8)[at, :, 5] = far.to(sr.E4M3).view(torch.uint8)
    v.view(torch.uint8)[at, :, 5] = 1                                               # 2^-9 of a unit of 2^-7
    q = torch.randn(count * new, h, dim, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    q[..., 0] = 8.0
    got = gn.attention_cached(q, *cache.args())
    check(q, cache, got, 2.0 ** -32, f"{above} above")


@pytest.mark.parametrize("keys", [2 ** 24 + 1001, 2 ** 25 + 130, 2 ** 27 + 777, 2 ** 30 - 300])
@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_distances_in_very_long_sequences(new, keys, dtype):
    """Where fp32 no longer holds every place, neighbouring keys still are one apart."""
    gen = torch.Generator("cuda").manual_seed(new)
    h, dim, page, near = 4, 16, 256, 2048
    own = near // page + 1                                     # the last pages are their own, all others one
    pools = [torch.randn(own + 1, 1, page, dim, generator=gen, device="cuda").mul(64.0).clamp(-448, 448).to(sr.E4M3).transpose(1, 2)
             for _ in "kv"]
    scales = [torch.full((own + 1, 1), 2.0 ** -6, device="cuda") for _ in "kv"]
    width = (keys + page - 1) // page
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, -own:] = torch.arange(1, own + 1, device="cuda")
    lengths = torch.tensor([keys], dtype=torch.int32, device="cuda")
    slopes = torch.tensor([0.5, 0.25, 1.0, 2.0], device="cuda")
    q = torch.randn(new, h, dim, generator=gen, device="cuda").to(dtype)
    out, got = gn.attention_cached(q, *pools, *scales, table, lengths, slopes=slopes)
    # what lies further back than 2000 keys has less than e^(-0.25 x 1900) of the weight
    place = torch.arange(keys - near, keys, device="cuda")
    k, v = (p[table[0, place // page].long()][torch.arange(near), place % page, 0].float().double() * 2.0 ** -6
            for p in pools)
    at = torch.arange(keys - new, keys, device="cuda")
    gap = (at[:, None] - place).double()
    t = torch.einsum("nhd,kd->hnk", q.double(), k) / 4 - slopes.double()[:, None, None] * gap.abs()
    size = torch.einsum("nhd,kd->hnk", q.double().abs(), k.abs()) / 4
    t.masked_fill_(gap < 0, -math.inf)
    lse = torch.logsumexp(t, 2)
    p = torch.exp(t - lse[..., None])
    # scores of the keys that matter: those with more than 2^-40 of the weight
    worst = (U32 * (20 * size + 4 * t.abs() + 4)).masked_fill(p < 2.0 ** -40, 0.0).amax(2)
    drop = 2.0 ** -17 * q.double().abs().amax(2).T * k.abs().sum(1).amax() / 4
    rel = 2 * worst + 2.0 ** -14
    br.check(got, lse, rel + drop + 4 * U32 * lse.abs(), "lse")
    want, absout = (torch.einsum("hnk,kd->nhd", p, x) for x in (v, v.abs()))
    u, low = br.half_step(dtype), br.least(dtype)
    off = low + u * want.abs() + (u + rel + 2 * drop).T[..., None] * absout + 2.0 ** -32 * near * v.abs().amax()
    br.check(out, want, off, "out")
