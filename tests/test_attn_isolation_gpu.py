"""What lies at tokens that a query (or key) does not see has no influence on
its results, to the last bit, whatever the scores are made of: infinities and
NaN, huge scores, several documents that hold such values around one that
does not, capped and biased scores, prefix masks, few and many queries."""
import math

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


def attend(t, cu_q, cu_k, prefix=None, backward=True, **how):
    how = dict(how, prefix=i32(prefix))
    out, lse = gn.attention_packed(t["q"], t["k"], t["v"], i32(cu_q), i32(cu_k), **how)
    got = dict(out=out, lse=lse)
    if backward:
        grads = gn.attention_packed_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, i32(cu_q), i32(cu_k), **how)
        got |= dict(zip(("dq", "dk", "dv"), grads))
    torch.cuda.synchronize()
    return got


def tensors(tq, tk, h, hk, dim, dtype, scale=1.0):
    return dict(q=rand((tq, h, dim), dtype, 1, scale), k=rand((tk, hk, dim), dtype, 2, scale), v=rand((tk, hk, dim), dtype, 3),
                dout=rand((tq, h, dim), dtype, 4))


def same_at(got, clean, queries, keys):
    """The results of these queries and keys have the same bits."""
    for name, t in got.items():
        for lo, hi in keys if name in ("dk", "dv") else queries:
            part = (lambda x: x[:, lo:hi]) if name == "lse" else (lambda x: x[lo:hi])
            a, b = part(t), part(clean[name])
            assert torch.equal(a, b), (name, lo, hi, int((a != b).sum()), int(torch.isnan(a.float()).sum()))


HOW = [dict(), dict(cap=20.0), dict(bias=True), dict(cap=20.0, bias=True), dict(cap=2.0, causal=True, prefix=[40, 3, 17]),
       dict(causal=True), dict(cap=30.0, bias=True, causal=True, prefix=[0, 90, 2])]


def spread(how, h):
    how = dict(how)
    if how.pop("bias", False):
        how["slopes"] = 2.0 ** -torch.arange(1, h + 1, device="cuda").float()
    return how


def with_bad(t, what, value, docs):
    """A copy whose tensors named in `what` hold value and -value at tokens `docs[name]`."""
    bad = {n: x.clone() for n, x in t.items()}
    for n in what:
        for lo, hi in docs[n]:
            bad[n][lo:hi:2] = value
            bad[n][lo + 1:hi:2] = -value
    return bad


CU_Q, CU_K = [3, 60, 261, 300], [5, 90, 291, 330]
MIDDLE = dict(q=((0, 3), (60, 261), (300, 310)), dout=((0, 3), (60, 261), (300, 310)),
              k=((0, 5), (90, 291), (330, 340)), v=((0, 5), (90, 291), (330, 340)))


@pytest.mark.parametrize("how", range(len(HOW)))
@pytest.mark.parametrize("h,hk,dim,dtype", [(2, 1, 64, BF), (4, 4, 128, FP), (8, 1, 40, BF)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nothing_infinite_reaches_other_documents(how, h, hk, dim, dtype, value):
    """One document (and what belongs to none) full of them: the other two stay finite."""
    how = spread(HOW[how], h)
    t = tensors(310, 340, h, hk, dim, dtype)
    for what in (("q",), ("k",), ("v",), ("dout",), ("q", "k", "v", "dout")):
        got = attend(with_bad(t, what, value, MIDDLE), CU_Q, CU_K, **how)
        for name, x in got.items():
            for lo, hi in ((5, 90), (291, 330)) if name in ("dk", "dv") else ((3, 60), (261, 300)):
                part = x[:, lo:hi] if name == "lse" else x[lo:hi]
                assert torch.isfinite(part.float()).all(), (name, what, lo)


@pytest.mark.parametrize("how", range(len(HOW)))
@pytest.mark.parametrize("h,hk,dim,dtype", [(2, 1, 64, BF), (4, 4, 128, FP), (8, 1, 40, BF)])
@pytest.mark.parametrize("value", [math.nan, math.inf, 3e4, 0.0])
def test_other_documents_keep_their_bits(how, h, hk, dim, dtype, value):
    how = spread(HOW[how], h)
    t = tensors(310, 340, h, hk, dim, dtype)
    clean = attend(t, CU_Q, CU_K, **how)
    for what in (("q",), ("k",), ("v",), ("dout",), ("q", "k", "v", "dout")):
        got = attend(with_bad(t, what, value, MIDDLE), CU_Q, CU_K, **how)
        same_at(got, clean, ((3, 60), (261, 300)), ((5, 90), (291, 330)))


@pytest.mark.parametrize("scale", [1.0, 4.0, 30.0])
@pytest.mark.parametrize("cap", [1.5, 25.0])
def test_capped_scores_on_both_sides_of_the_formulas(scale, cap):
    """Small and large scores in one tile against the formulas."""
    cu = [0, 150, 400]
    t = tensors(400, 400, 4, 2, 64, BF)
    t["q"][::3] *= scale
    t["k"][::2] *= scale
    how = dict(cap=cap, causal=True, prefix=[50, 0])
    got = attend(t, cu, cu, **how)
    for name, (value, bound) in br.attention(t["q"], t["k"], t["v"], cu, cu, dout=t["dout"], **how).items():
        br.check(got[name], value, bound, name)


@pytest.mark.parametrize("how", [dict(), dict(cap=20.0), dict(cap=9.0, bias=True), dict(causal=True)])
@pytest.mark.parametrize("h,hk,dim,dtype,lens", [(4, 1, 64, BF, [1, 3, 2, 2, 1]), (8, 2, 128, FP, [3, 1, 1, 3, 1]), (16, 1, 40, BF, [1, 3, 2, 2, 2]),
                                                 (24, 1, 128, BF, [1, 3, 2, 2, 2]), (8, 8, 64, BF, [2, 4, 8, 1, 5])])
@pytest.mark.parametrize("value", [math.nan, math.inf, 50.0])
def test_few_queries_of_several_documents(h, hk, dim, dtype, lens, how, value):
    """Documents that share a tile of few rows: every other one's keys hold such values."""
    how = spread(how, h)
    k_lens = [333, 200, 61, 700, 150]
    cu_q, cu_k = ([sum(n[:i]) for i in range(6)] for n in (lens, k_lens))
    t = tensors(cu_q[-1], cu_k[-1], h, hk, dim, dtype)
    clean = attend(t, cu_q, cu_k, backward=False, **how)
    for first in (0, 1):
        docs = tuple((cu_k[d], cu_k[d + 1]) for d in range(first, 5, 2))
        keep = tuple((cu_q[d], cu_q[d + 1]) for d in range(1 - first, 5, 2))
        for what in (("k",), ("v",), ("k", "v")):
            got = attend(with_bad(t, what, value, dict(k=docs, v=docs)), cu_q, cu_k, backward=False, **how)
            same_at(got, clean, keep, ())


@pytest.mark.parametrize("how", [dict(), dict(cap=20.0), dict(cap=9.0, bias=True)])
@pytest.mark.parametrize("h,hk,dim,dtype,new", [(4, 1, 64, BF, 4), (16, 2, 128, FP, 4), (16, 4, 128, BF, 2), (32, 2, 64, BF, 4)])
@pytest.mark.parametrize("value", [math.nan, math.inf, 40.0])
def test_new_tokens_do_not_see_each_others_keys_ahead(h, hk, dim, dtype, new, how, value):
    """The last token's key and value change: the tokens before it in the same tile keep their bits."""
    how = dict(spread(how, h), causal=True)
    cu_q, cu_k = [0, new, 2 * new], [0, 300, 1000]
    t = tensors(cu_q[-1], cu_k[-1], h, hk, dim, dtype, scale=1.5)
    clean = attend(t, cu_q, cu_k, backward=False, **how)
    for what in (("k",), ("v",), ("k", "v")):
        last = ((299, 300), (999, 1000))
        got = attend(with_bad(t, what, value, dict(k=last, v=last)), cu_q, cu_k, backward=False, **how)
        same_at(got, clean, ((0, new - 1), (new, 2 * new - 1)), ())


@pytest.mark.parametrize("how", range(len(HOW)))
@pytest.mark.parametrize("h,hk,dim,dtype", [(2, 1, 64, BF), (3, 3, 128, FP), (8, 1, 24, BF)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_documents_between_two_that_hold_such_values(how, h, hk, dim, dtype, value):
    """The first and the last of three hold them, and the middle one none."""
    how = spread(HOW[how], h)
    cu_q, cu_k = [0, 37, 90, 222], [0, 41, 111, 280]
    t = tensors(222, 280, h, hk, dim, dtype)
    clean = attend(t, cu_q, cu_k, **how)
    docs = dict(q=((0, 37), (90, 222)), dout=((0, 37), (90, 222)), k=((0, 41), (111, 280)), v=((0, 41), (111, 280)))
    for what in (("q",), ("k",), ("v",), ("dout",), ("q", "k", "v", "dout")):
        same_at(attend(with_bad(t, what, value, docs), cu_q, cu_k, **how), clean, ((37, 90),), ((41, 111),))


@pytest.mark.parametrize("h,hk,dim,dtype", [(2, 1, 64, BF), (4, 4, 128, FP)])
@pytest.mark.parametrize("how", [dict(), dict(cap=6.0, bias=True)])
def test_a_document_of_nan_throughout(h, hk, dim, dtype, how):
    """Values or gradients that are NaN everywhere in a document give NaN everywhere
    there, its lse stays, and so do the two documents beside it."""
    cu = [0, 50, 700, 740]
    t = tensors(740, 740, h, hk, dim, dtype)
    for causal in (False, True):
        own = dict(spread(how, h), causal=causal)
        clean = attend(t, cu, cu, **own)
        for name, shows in (("v", ("out", "dq", "dk")), ("dout", ("dq", "dk", "dv"))):
            bad = {n: x.clone() for n, x in t.items()}
            bad[name][50:700] = math.nan
            got = attend(bad, cu, cu, **own)
            assert torch.equal(got["lse"], clean["lse"])
            same_at(got, clean, ((0, 50), (700, 740)), ((0, 50), (700, 740)))
            for what in shows:
                assert torch.isnan(got[what][50:700].float()).all(), (name, what)
        few = attend(dict(bad, q=t["q"][:9], v=torch.where(torch.arange(740, device="cuda")[:, None, None] < 700, math.nan, t["v"])),
                     [0, 3, 6, 9], cu, backward=False, **own)
        kept = attend(dict(t, q=t["q"][:9]), [0, 3, 6, 9], cu, backward=False, **own)
        assert torch.isnan(few["out"][:6].float()).all() and torch.equal(few["out"][6:], kept["out"][6:])
        assert torch.equal(few["lse"], kept["lse"])


@pytest.mark.parametrize("h,hk,dim,dtype", [(2, 1, 64, BF), (4, 4, 128, FP)])
@pytest.mark.parametrize("how", [dict(), dict(cap=6.0, bias=True)])
def test_what_sees_such_a_value_shows_it(h, hk, dim, dtype, how):
    """One value row, key row, query row or gradient row at a time, of a causal document between two clean ones."""
    how = dict(spread(how, h), causal=True)
    cu, at = [0, 50, 300, 340], 200
    t = tensors(340, 340, h, hk, dim, dtype)
    clean = attend(t, cu, cu, **how)
    for name, shows in (("v", {"out": (at, 300), "dq": (at, 300)}), ("k", {"out": (at, 300), "dq": (at, 300)}),
                        ("q", {"out": (at, at + 1), "dk": (50, at + 1), "dv": (50, at + 1), "dq": (at, at + 1)}),
                        ("dout", {"dq": (at, at + 1), "dk": (50, at + 1), "dv": (50, at + 1)})):
        bad = {n: x.clone() for n, x in t.items()}
        bad[name][at] = math.nan
        got = attend(bad, cu, cu, **how)
        for what, (lo, hi) in shows.items():
            assert torch.isnan(got[what][lo:hi].float()).all(), (name, what)
            assert torch.equal(got[what][:50], clean[what][:50]) and torch.equal(got[what][300:], clean[what][300:]), (name, what)
            if what in ("out", "dq"):
                assert torch.equal(got[what][50:lo], clean[what][50:lo]), (name, what)
