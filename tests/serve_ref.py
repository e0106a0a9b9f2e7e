"""RMS norm and the paged cache in 8 bits from their definitions in 64 bits, and how
far a kernel may be from them (as in tests/block_ref.py: every rounding half a
step, carried through the formulas)."""
import math

import torch

from tests import block_ref as br

U32 = br.U32
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -100           # the smallest scale of a page


# ---------------------------------------------------------------------------
# RMS norm: (value, bound) of each output
# ---------------------------------------------------------------------------
def rms_norm(x, w, eps, residual=None, dy=None, dtotal=None):
    """Of two-dimensional rows.  The 8-bit output's bound is on byte times scale."""
    u, low = br.half_step(x.dtype), br.least(x.dtype)
    total = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    t = total.double()
    n = t.shape[1]
    rstd = 1.0 / torch.sqrt((t * t).mean(1, keepdim=True) + eps)
    wd = w.double() if w is not None else torch.ones(n, dtype=torch.float64, device=x.device)
    steps = 128 * U32                     # a thread's elements, the warp's and the CTA's sums
    y = t * rstd * wd
    r = {"total": (total.double(), torch.zeros_like(t)), "rstd": (rstd[:, 0], steps * rstd[:, 0]),
         "y": (y, low + (u + steps + 4 * U32) * y.abs())}
    most = y.abs().amax(1, keepdim=True)
    r["scales"] = (most[:, 0] / 448, (steps + 4 * U32) * most[:, 0] / 448)
    # half a step of e4m3, of its subnormals (2^-9 scale), and what fp32 flushes
    r["y8"] = (y, (2.0 ** -4 + 2 * steps) * y.abs() + (2.0 ** -10 + 1e-30) * most / 448)
    if dy is not None:
        g0 = dy.double()
        g = g0 * wd
        along = (g * t).sum(1, keepdim=True) / n
        dx = rstd * g - t * rstd ** 3 * along
        off = 3 * steps * (rstd * g.abs() + t.abs() * rstd ** 3 * (g * t).abs().mean(1, keepdim=True))
        if dtotal is not None:
            dx = dx + dtotal.double()
        r["dx"] = (dx, low + (u + 2 * U32) * dx.abs() + off)
        if w is not None:
            dw = (g0 * t * rstd).sum(0)
            chain = (t.shape[0] + 64) * U32        # at worst one chain over the rows
            r["dw"] = (dw, br.least(w.dtype) + br.half_step(w.dtype) * dw.abs()
                       + (chain + steps) * (g0 * t * rstd).abs().sum(0))
    return r


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
def cast_e4m3(x):
    """fp64 values on e4m3's grid, ties to even, past 448 to 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def least_scale(most):
    """The least power of two >= 2^-100 of which 448 times is no less (a number)."""
    if not math.isfinite(most):
        return math.nan
    e = -100
    if most > 0:
        m, x = math.frexp(most)                   # m in [1/2, 1); 448 = 0.875 2^9
        e = max(e, x - 9 + (m > 0.875))
    return 2.0 ** e


class Cache:
    """A cache whose sequences hold `lens` tokens, in pages from anywhere in the pool;
    what no sequence owns holds NaN bytes and NaN scales."""

    def __init__(self, lens, page, hk, dim, seed=0, order="heads", device="cuda", spare=2, width=None, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.page = list(lens), page
        wants = [(n + page - 1) // page for n in lens]
        pages = sum(wants) + spare
        places = torch.randperm(pages, generator=gen).tolist()
        width = width or max(1, max(wants))
        table = torch.full((len(self.lens), width), -1, dtype=torch.int32)
        at = 0
        for s, want in enumerate(wants):
            table[s, :want] = torch.tensor(places[at:at + want], dtype=torch.int32)
            at += want
        self.table_host = table.tolist()
        self.table = table.to(device)
        self.lengths = torch.tensor(self.lens, dtype=torch.int32, device=device)
        shape = dict(heads=(pages, hk, page, dim), tokens=(pages, page, hk, dim), slots=(page, hk, pages, dim))[order]
        for name in "kv":
            buf = torch.full(shape, 0x7f, dtype=torch.uint8, device=device)
            pool = dict(heads=buf.transpose(1, 2), tokens=buf, slots=buf.permute(2, 0, 1, 3))[order] if order != "tokens" else buf
            setattr(self, name + "_bytes", pool)
            setattr(self, name + "_pages", pool.view(E4M3))
            setattr(self, name + "_scales", torch.full((pages, hk), math.nan, device=device))
        for s, n in enumerate(self.lens):
            for p in range(wants[s]):
                held, page_at = min(page, n - p * page), self.table_host[s][p]
                for name in "kv":
                    x = torch.randn(held, hk, dim, generator=gen) * 1.5 * 2.0 ** (spread * torch.randn(1, hk, 1, generator=gen))
                    scale = torch.tensor([least_scale(float(v)) for v in x.abs().amax(dim=(0, 2))])
                    self.pages(name)[page_at, :held] = (x / scale[:, None]).to(E4M3).view(torch.uint8).to(device)
                    self.scales(name)[page_at] = scale.to(device)

    def pages(self, name):
        return getattr(self, name + "_bytes")

    def scales(self, name):
        return getattr(self, name + "_scales")

    def args(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales, self.table, self.lengths

    def copy(self):
        other = Cache.__new__(Cache)
        other.__dict__.update(self.__dict__)
        for name in "kv":
            b = self.pages(name).clone(memory_format=torch.preserve_format)
            setattr(other, name + "_bytes", b)
            setattr(other, name + "_pages", b.view(E4M3))
            setattr(other, name + "_scales", self.scales(name).clone())
        return other

    def values(self, name, s):
        """Sequence s' tokens in 64 bits, [length, Hk, D]."""
        n, page = self.lens[s], self.page
        hk, dim = self.pages(name).shape[2:]
        out = torch.zeros(n, hk, dim, dtype=torch.float64, device=self.table.device)
        for p in range((n + page - 1) // page):
            at, held = self.table_host[s][p], min(page, n - p * page)
            if 0 <= at < self.pages(name).shape[0]:
                values = self.pages(name)[at, :held].view(E4M3).double()
                out[p * page:p * page + held] = values * self.scales(name)[at].double()[:, None]
        return out


def attention(q, cache, cu, causal=True, slopes=None, cap=0.0, scale=None):
    """{name: (value, bound)} of attention over a Cache; cu a list."""
    k = torch.cat([cache.values("k", s) for s in range(len(cache.lens))])
    v = torch.cat([cache.values("v", s) for s in range(len(cache.lens))])
    ends = [0]
    for n in cache.lens:
        ends.append(ends[-1] + n)
    r = br.attention(q, k, v, cu, ends, causal=causal, slopes=slopes, cap=cap, scale=scale)
    # The query's split drops less than 2^-17 of its largest channel from a channel;
    # the weights' drops at most 2^-18 of the largest weight from a weight, and keeps
    # 2^-9 of each (which the half format's step covers in bf16, and 2^-11 in fp16).
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, off = r["out"]
    for s in range(len(cache.lens)):
        rows, keys = slice(cu[s], cu[s + 1]), slice(ends[s], ends[s + 1])
        if rows.start == rows.stop or keys.start == keys.stop:
            continue
        for h in range(heads):
            kh, vh = k[keys, h // group], v[keys, h // group]
            drop = 2.0 ** -17 * q[rows, h].double().abs().amax(1) * kh.abs().sum(1).amax() * abs(scale)
            off[rows, h] += (2 * drop[:, None] + 2.0 ** -18) * vh.abs().sum(0)
            r["lse"][1][h, rows] += drop
    return r
