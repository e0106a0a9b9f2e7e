"""The transformer-block operators from their definitions in 64 bits, and how
far a kernel may be from them: every rounding of the kernels' (half a step,
finfo.eps / 2, each; half a step of the subnormals below the normal range)
carried through the formulas.  fp32 chains count one 2^-24 per step."""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half a step of the subnormals, and what fp32 flushes to zero on the way."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2 + 2.0 ** -126


def outside(got, want, bound):
    """How many elements are further from `want` than `bound` allows (a NaN
    where none belongs is one); infinities have to be equal."""
    got, want, bound = got.double(), want.double(), torch.as_tensor(bound, dtype=torch.float64, device=want.device)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    return int((~(same | ((got - want).abs() <= bound))).sum())


def check(got, want, bound, what):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = outside(got, want, bound)
    err = (got.double() - want).abs().nan_to_num(math.inf, math.inf)
    assert bad == 0, f"{what}: {bad} of {want.numel()} outside the bound, max error {float(err.max()):.3e}"


# ---------------------------------------------------------------------------
# layer norm: (value, bound) of each output
# ---------------------------------------------------------------------------
def layer_norm(x, w, b, eps, dy=None):
    u, steps = half_step(x.dtype), 128      # a thread's elements, the warp's and the CTA's sums: under 128 steps
    xd = x.double()
    n = xd.shape[1]
    mean = xd.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((xd - mean) ** 2).mean(1, keepdim=True) + eps)
    hat = (xd - mean) * rstd
    one = torch.ones(n, dtype=torch.float64, device=x.device)
    wd = w.double() if w is not None else one
    bd = b.double() if b is not None else 0 * one
    y = hat * wd + bd
    size = xd.abs().amax(1, keepdim=True) * rstd             # |x| in units of the standard deviation
    e = steps * U32 * (1 + size)                             # error of hat over max(1, |hat|)
    hats = 1 + hat.abs()
    low = least(x.dtype)
    r = {"y": (y, low + u * y.abs() + e * (hats * wd.abs() + bd.abs())),
         "mean": (mean[:, 0], steps * U32 * xd.abs().amax(1)),
         "rstd": (rstd[:, 0], e[:, 0] * rstd[:, 0] * (1 + size[:, 0]))}
    if dy is not None:
        g0 = dy.double()
        g = g0 * wd
        m0, m1 = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
        dx = rstd * (g - m0 - hat * m1)
        spread = g.abs() + g.abs().mean(1, keepdim=True) + hats * (g.abs() * hats).mean(1, keepdim=True)
        r["dx"] = (dx, low + u * dx.abs() + 3 * e * rstd * spread * (1 + size))
        if w is not None:
            uw = half_step(w.dtype)
            chain = (xd.shape[0] + 64) * U32                 # at worst one chain over the rows
            dw, db = (g0 * hat).sum(0), g0.sum(0)
            r["dw"] = (dw, uw * dw.abs() + (g0.abs() * hats * (chain + e)).sum(0))
            r["db"] = (db, uw * db.abs() + chain * g0.abs().sum(0))
    return r


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope(x, positions, axes, theta, interleaved, inverse):
    angle = torch.cat([positions[:, n:n + 1].double() * theta ** (-torch.arange(0, d, 2, dtype=torch.float64,
                                                                                device=x.device) / d)
                       for n, d in enumerate(axes)], dim=1)[:, None, :]
    if inverse:
        angle = -angle
    half = angle.shape[-1]
    xd = x.double()
    y, size = xd.clone(), torch.zeros_like(xd)
    first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                     else (slice(0, half), slice(half, 2 * half)))
    a, b = xd[..., first], xd[..., second]
    y[..., first], y[..., second] = a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()
    size[..., first] = size[..., second] = a.abs() + b.abs()
    # the rest of a turn in fp32 (2 pi 2^-26 turns), sine and cosine (2 steps), products and sum (3)
    return y, (half_step(x.dtype) * y.abs() + least(x.dtype)) * (size > 0) + 12 * U32 * size


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def spans(tq, tk, cu_q, cu_k, causal, prefix):
    """[tq, tk] truth values: which keys a query sees; and the key each stands at."""
    seen = torch.zeros(tq, tk, dtype=torch.bool)
    stands = torch.zeros(tq, dtype=torch.float64)
    for d in range(len(cu_q) - 1):
        for i in range(cu_q[d], cu_q[d + 1]):
            at = cu_k[d + 1] - cu_q[d + 1] + i
            stands[i] = at
            hi = cu_k[d + 1]
            if causal:
                hi = min(hi, max(at + 1, cu_k[d] + (prefix[d] if prefix else 0)))
            seen[i, cu_k[d]:max(hi, cu_k[d])] = True
    return seen, stands


def attention(q, k, v, cu_q, cu_k, causal=False, prefix=None, slopes=None, cap=0.0, scale=None, dout=None):
    """{name: (value, bound)}; cu_q, cu_k and prefix are lists."""
    u, low = half_step(q.dtype), least(q.dtype)
    tq, h, dim = q.shape
    tk, hk, _ = k.shape
    scale = dim ** -0.5 if scale is None else scale
    seen, stands = spans(tq, tk, cu_q, cu_k, causal, prefix)
    seen, stands = seen.to(q.device), stands.to(q.device)
    far = (stands[:, None] - torch.arange(tk, device=q.device)[None]).abs()
    clean = lambda t: t.double()  # noqa: E731
    res = {n: (torch.zeros(s, dtype=torch.float64, device=q.device), torch.zeros(s, dtype=torch.float64, device=q.device))
           for n, s in (("out", q.shape), ("lse", (h, tq)), ("dq", q.shape), ("dk", k.shape), ("dv", k.shape))}
    # keys and queries that nobody sees hold whatever they hold
    used_k, used_q = seen.any(0)[:, None], seen.any(1)[:, None]
    for head in range(h):
        g = head * hk // h
        qh = torch.where(used_q, clean(q[:, head]), 0.0)
        kh, vh = (torch.where(used_k, clean(t[:, g]), 0.0) for t in (k, v))
        raw = qh @ kh.T * scale
        size = qh.abs() @ kh.abs().T * abs(scale)
        t = cap * torch.tanh(raw / cap) if cap else raw
        slack = 1 - torch.tanh(raw / cap) ** 2 if cap else torch.ones_like(raw)
        if slopes is not None:
            t = t - slopes[head].double() * far
        # error of a score: the dot product's chain, cap and bias, the change to base 2
        delta_t = U32 * ((dim + 4) * size + 8 * (cap or 0.0) + 4 * t.abs() + 4)
        t = t.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(t, 1)
        p = torch.where(seen, torch.exp(t - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
        worst = torch.where(seen, delta_t, 0.0).amax(1, keepdim=True) if tk else torch.zeros(tq, 1, device=q.device)
        rel = 2 * worst + 2.0 ** -20 + tk * U32 / 64         # of a weight: its own score's error and the sum's
        out = p @ vh
        absout = p @ vh.abs()
        res["out"][0][:, head], res["out"][1][:, head] = (
            out, low + u * out.abs() + (u + rel) * absout + low * (seen.double() @ vh.abs()))
        res["lse"][0][head] = lse
        res["lse"][1][head] = rel[:, 0] + 4 * U32 * lse.abs().nan_to_num(0, 0, 0)
        if dout is None:
            continue
        do = torch.where(used_q, clean(dout[:, head]), 0.0)
        dp = do @ vh.T
        delta = (do * out).sum(1, keepdim=True)
        ds = p * (dp - delta) * slack
        # delta comes from the rounded output, dp from an fp32 chain; ds is rounded once more
        d_delta = (do.abs() * res["out"][1][:, head]).sum(1, keepdim=True) + dim * U32 * (do * out).abs().sum(1, keepdim=True)
        d_dp = (dim + 4) * U32 * (do.abs() @ vh.abs().T)
        d_slack = 16 * U32 + 2 * delta_t / cap if cap else 0.0
        d_ds = u * ds.abs() + seen * low * (1 + (dp - delta).abs()) + p * (d_delta + d_dp + (rel + d_slack + 8 * U32) * (dp - delta).abs())
        res["dq"][0][:, head] = ds @ kh * scale
        res["dq"][1][:, head] = (d_ds + tk * U32 / 16 * ds.abs()) @ kh.abs() * abs(scale)
        res["dk"][0][:, g] += ds.T @ qh * scale
        res["dk"][1][:, g] += (d_ds + tq * U32 / 16 * ds.abs()).T @ qh.abs() * abs(scale)
        res["dv"][0][:, g] += p.T @ do
        res["dv"][1][:, g] += (p * (u + rel + tq * U32 / 16) + seen * low).T @ do.abs()
    for n in ("dq", "dk", "dv"):
        res[n] = (res[n][0], res[n][1] + u * res[n][0].abs() + low)
    return res if dout is not None else {n: res[n] for n in ("out", "lse")}
