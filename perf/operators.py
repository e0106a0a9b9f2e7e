"""The operators of a packed image transformer block, as they are measured.

Three operators around the residual-gate update that the package already has:

  layer norm   y = (x - mean) rstd w + b over the last axis, and its backward
               pass with the reductions of the weight's and the bias' gradient;
  rope         rotary positions over several axes (time, height, width, text)
               of the query and key heads, forward and inverse (its gradient);
  attention    of packed documents: every query sees a run of its own
               document's keys (all of them, the causal ones, or a prefix and
               the causal ones), scores optionally capped by a tanh and biased
               by the distance, with grouped key/value heads, forward,
               backward and for single new tokens.

With ``own`` false, ``run`` evaluates the formulas with elementary torch
operations in fp32; with ``own`` true it calls the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the norm ahead of a modulation (no weight of its own), one new token
        dict(name="norm_one_token", op="norm", rows=1, cols=6144, type="bf16", weight="none", train=False),
        # the same width over the 4096 image and 512 text tokens of a 1024 x 1024 image, in a training step
        dict(name="norm_train_image", op="norm", rows=4608, cols=6144, type="bf16", weight="fp32", train=True),
        # the norm of every query head ahead of the rotation: very many short rows
        dict(name="norm_train_heads", op="norm", rows=110592, cols=128, type="fp16", weight="fp16", train=True),
        # odd width and row count in full precision, rows cut out of a wider tensor
        dict(name="norm_train_odd", op="norm", rows=3001, cols=1003, type="fp32", weight="fp32", train=True),
        # one new token's query and key heads
        dict(name="rope_one_token", op="rope", tokens=1, heads=48, kv_heads=8, dim=128, axes="32,32,32,32",
             theta=2000.0, positions="image", interleaved=True, inverse=False, type="bf16"),
        # four-axis positions of a 1024 x 1024 image and its text, query and key heads
        dict(name="rope_image", op="rope", tokens=4608, heads=48, kv_heads=48, dim=128, axes="32,32,32,32",
             theta=2000.0, positions="image", interleaved=True, inverse=False, type="bf16"),
        # the gradient through the rotation of video tokens (fractional times), halves paired, an unrotated rest
        dict(name="rope_video_gradient", op="rope", tokens=30030, heads=12, kv_heads=3, dim=128, axes="24,36,36",
             theta=10000.0, positions="video", interleaved=False, inverse=True, type="fp32"),
        # one new token for each of many ragged sequences, grouped heads
        dict(name="attn_one_token", op="attn", q_lens="1," * 23 + "1",
             k_lens="8000,17,3501,1,6007,129,4096,777,2048,5555,64,7013,333,1000,4999,2500,1,6500,88,3030,7777,15,450,5120",
             heads=32, kv_heads=8, dim=128, causal=True, prefix="", cap=0.0, bias=False, type="bf16", train=False),
        # images of several sizes with their texts packed into one call, every token sees its own image's
        dict(name="attn_images", op="attn", q_lens="4608,1536,2111,300", k_lens="4608,1536,2111,300",
             heads=24, kv_heads=24, dim=128, causal=False, prefix="", cap=0.0, bias=False, type="bf16", train=False),
        # a training step over packed images
        dict(name="attn_train_images", op="attn", q_lens="4608,1536,1500,548", k_lens="4608,1536,1500,548",
             heads=24, kv_heads=24, dim=128, causal=False, prefix="", cap=0.0, bias=False, type="bf16", train=True),
        # a training step over texts whose prompts are seen whole, capped scores, grouped narrow heads
        dict(name="attn_train_prefix", op="attn", q_lens="1500,37,2222,1,600", k_lens="1500,37,2222,1,600",
             heads=16, kv_heads=4, dim=64, causal=True, prefix="700,37,5,0,100", cap=50.0, bias=False,
             type="fp16", train=True),
        # one long causal sequence with a distance bias and an uncommon head width
        dict(name="attn_long_bias", op="attn", q_lens="16384", k_lens="16384", heads=8, kv_heads=8, dim=96,
             causal=True, prefix="", cap=0.0, bias=True, type="bf16", train=False),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    if op == "norm":
        cols = _log(rng, 32, 12288)
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        kind = rng.choice(["bf16", "fp16", "fp32"])
        return dict(op="norm", rows=_log(rng, 1, min(200000, 28_000_000 // cols)), cols=cols, type=kind,
                    weight=rng.choice(["none", "fp32", kind]), train=rng.random() < 0.6)
    if op == "rope":
        axes = rng.choice(["32,32,32,32", "16,56,56", "24,36,36", "44,42,42", "64", "20,22,22", "16,24,24"])
        width = sum(int(a) for a in axes.split(","))
        kv_heads = rng.choice([1, 2, 3, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 6])
        dim = width + rng.choice([0, 0, 8, 32])
        return dict(op="rope", tokens=_log(rng, 1, min(60000, 100_000_000 // (dim * (heads + kv_heads)))), heads=heads,
                    kv_heads=kv_heads, dim=dim, axes=axes, theta=rng.choice([2000.0, 10000.0, 1000000.0]),
                    positions=rng.choice(["image", "video"]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.4, type=rng.choice(["bf16", "fp16", "fp32"]))
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 8])
    dim = rng.choice([64, 64, 128, 128, 96, 80, 72, 40])
    causal = rng.random() < 0.6
    docs = _log(rng, 1, 24)
    common = dict(heads=heads, kv_heads=kv_heads, dim=dim, causal=causal, cap=rng.choice([0.0, 0.0, 30.0]),
                  bias=rng.random() < 0.3, type=rng.choice(["bf16", "fp16"]))
    if rng.random() < 0.3:                       # new tokens: one for each document, or a few
        new = rng.choice([1, 1, 1, 2, 4])
        k_lens = [_log(rng, new, 8192) for _ in range(docs)]
        return dict(op="attn", q_lens=",".join([str(new)] * docs), k_lens=_text(k_lens), prefix="", train=False,
                    **common)
    total = _log(rng, max(24, 8 * docs), 6000 if heads <= 16 else 3000)
    cuts = sorted(rng.randint(0, total) for _ in range(docs - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    prefix = _text([rng.randint(0, n) for n in lens]) if causal and rng.random() < 0.5 else ""
    return dict(op="attn", q_lens=_text(lens), k_lens=_text(lens), prefix=prefix, train=rng.random() < 0.5, **common)


def _text(numbers):
    return ",".join(str(n) for n in numbers)


def _numbers(text):
    return [int(t) for t in text.split(",")] if text else []


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = TYPES[case["type"]]

    def normal(*shape, scale=1.0, to=kind):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    state = dict(case)
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # channels of a residual stream: their own offsets, a few of them large; rows of a wider tensor
        offset = normal(cols, scale=0.5, to=torch.float32)
        offset[:: max(1, cols // 3)] *= 20.0
        wide = (torch.randn((rows, cols + 16), generator=gen, device="cuda") * 2.0)
        state["x"] = (wide[:, 8:8 + cols] + offset).to(kind)
        if cols % 8:
            state["x"] = torch.cat([state["x"], state["x"][:, :5]], dim=1)[:, :cols]   # a row stride of its own
        if case["weight"] != "none":
            wkind = TYPES[case["weight"]]
            state["w"] = normal(cols, scale=0.2, to=torch.float32).add_(1.0).to(wkind)
            state["b"] = normal(cols, scale=0.2, to=wkind)
        if case["train"]:
            state["dy"] = normal(rows, cols)
    elif case["op"] == "rope":
        t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        qkv = normal(t, h + 2 * g, d)                         # the fused projection of a block
        state["q"], state["k"] = qkv[:, :h], qkv[:, h:h + g]
        axes = len(_numbers(case["axes"]))
        token = torch.arange(t, device="cuda") + int(torch.randint(0, 1000, (), generator=gen, device="cuda"))
        if case["positions"] == "image":                      # whole positions: rows and columns of a 64-wide grid
            parts = [token // 4096, token // 64 % 64, token % 64, token]
            state["positions"] = torch.stack(parts[:axes], dim=1).to(torch.int32)
        else:                                                 # frames at fractional times, far into a video
            parts = [token // 1560 * (16 / 25) + 100000.0, token // 52 % 30, token % 52, token]
            state["positions"] = torch.stack([p.double() for p in parts[:axes]], dim=1).float()
    else:
        q_lens, k_lens = _numbers(case["q_lens"]), _numbers(case["k_lens"])
        tq, tk, h, g, d = sum(q_lens), sum(k_lens), case["heads"], case["kv_heads"], case["dim"]
        if case["q_lens"] == case["k_lens"]:                  # slices of the fused projection
            qkv = torch.cat([normal(tq, h + g, d, scale=1.4), normal(tq, g, d)], dim=1)
            state["q"], state["k"], state["v"] = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        else:                                                 # a cache of keys and values beside new queries
            state["q"], state["k"], state["v"] = (normal(tq, h, d, scale=1.4), normal(tk, g, d, scale=1.4),
                                                  normal(tk, g, d))
        state["cu_q"] = _ends(q_lens)
        state["cu_k"] = _ends(k_lens)
        state["prefix"] = (torch.tensor(_numbers(case["prefix"]), dtype=torch.int32, device="cuda")
                           if case["prefix"] else None)
        state["slopes"] = (torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda", dtype=torch.float32) / h)
                           if case["bias"] else None)
        if case["train"]:
            state["dout"] = normal(tq, h, d)
    return state


def _ends(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
EPS = 1e-6


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[state["op"]](state)


def _run_own(s):
    import channels_last_groupnorm_gb300 as gn

    if s["op"] == "norm":
        y, mean, rstd = gn.layer_norm(s["x"], s.get("w"), s.get("b"), eps=EPS)
        if not s["train"]:
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = gn.layer_norm_backward(s["dy"], s["x"], mean, rstd, s.get("w"))
        return _some(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)
    if s["op"] == "rope":
        q, k = gn.rope_nd(s["q"], s["k"], s["positions"], _numbers(s["axes"]), theta=s["theta"],
                          interleaved=s["interleaved"], inverse=s["inverse"])
        return {"q": q, "k": k}
    how = dict(causal=s["causal"], prefix=s["prefix"], slopes=s["slopes"], cap=s["cap"])
    out, lse = gn.attention_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], **how)
    if not s["train"]:
        return {"out": out, "lse": lse}
    dq, dk, dv = gn.attention_packed_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"], **how)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(dim=1)
    centred = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((centred * centred).mean(dim=1) + EPS)
    hat = centred * rstd[:, None]
    y = hat
    if "w" in s:
        y = hat * s["w"].float() + s["b"].float()
    y = y.to(s["x"].dtype)
    if not s["train"]:
        return {"y": y, "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    g = dy * s["w"].float() if "w" in s else dy
    dx = rstd[:, None] * (g - g.mean(dim=1, keepdim=True) - hat * (g * hat).mean(dim=1, keepdim=True))
    dw = (dy * hat).sum(dim=0).to(s["w"].dtype) if "w" in s else None
    db = dy.sum(dim=0).to(s["w"].dtype) if "w" in s else None
    return _some(y=y, mean=mean, rstd=rstd, dx=dx.to(s["x"].dtype), dw=dw, db=db)


def _plain_rope(s):
    axes = _numbers(s["axes"])
    # the axis of every pair of channels and the pair's place among its axis' pairs
    pairs = torch.tensor([a // 2 for a in axes], device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(axes), device="cuda"), pairs)
    place = torch.arange(axis.numel(), device="cuda") - (pairs.cumsum(0) - pairs)[axis]
    # angles in 64 bits: far positions lose their phase in 32
    rate = torch.exp(-math.log(s["theta"]) * place.double() / pairs[axis].double())
    angle = (s["positions"].double()[:, axis] * rate)[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if s["inverse"]:
        sin = -sin
    return {"q": _turned(s["q"], cos, sin, s["interleaved"]), "k": _turned(s["k"], cos, sin, s["interleaved"])}


def _turned(x, cos, sin, interleaved):
    half = cos.shape[-1]
    f = x[..., :2 * half].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if interleaved else (f[..., :half], f[..., half:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return torch.cat([y.to(x.dtype), x[..., 2 * half:]], dim=-1)


def _places(count, ends):
    """The document of each of `count` tokens, and the token's place in it."""
    token = torch.arange(count, device="cuda")
    doc = (token[:, None] >= ends[1:][None, :]).sum(dim=1)
    return doc, token - ends[doc]


def _plain_attn(s):
    q, k, v = (s[n].float().transpose(0, 1) for n in "qkv")              # [heads, tokens, dim]
    group = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(group, dim=0), v.repeat_interleave(group, dim=0)
    scale = 1.0 / math.sqrt(q.shape[-1])
    q_doc, q_place = _places(q.shape[1], s["cu_q"])
    k_doc, k_place = _places(k.shape[1], s["cu_k"])
    new = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])
    place = (q_place + new[q_doc])[:, None]                              # the last query stands at the last key
    seen = q_doc[:, None] == k_doc[None, :]
    if s["causal"]:
        early = k_place[None, :] <= place
        if s["prefix"] is not None:
            early = early | (k_place < s["prefix"][k_doc])[None, :]
        seen = seen & early
    scores = torch.matmul(q, k.transpose(1, 2)) * scale
    if s["cap"]:
        bent = torch.tanh(scores / s["cap"])
        scores = bent * s["cap"]
    if s["slopes"] is not None:
        scores = scores - s["slopes"][:, None, None] * (place - k_place[None, :]).abs().float()
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.max(dim=2, keepdim=True).values
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    del scores
    total = p.sum(dim=2, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v)
    kind = s["q"].dtype
    result = {"out": out.transpose(0, 1).to(kind), "lse": lse}
    if not s["train"]:
        return result
    dout = s["dout"].float().transpose(0, 1)
    dv = torch.matmul(p.transpose(1, 2), dout)
    dp = torch.matmul(dout, v.transpose(1, 2))
    ds = p * (dp - (p * dp).sum(dim=2, keepdim=True))
    if s["cap"]:
        ds = ds * (1.0 - bent * bent)
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(1, 2), q) * scale
    heads = (k.shape[0] // group, group)
    result["dq"] = dq.transpose(0, 1).to(kind)
    result["dk"] = dk.unflatten(0, heads).sum(dim=1).transpose(0, 1).to(kind)
    result["dv"] = dv.unflatten(0, heads).sum(dim=1).transpose(0, 1).to(kind)
    return result


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "norm":
        n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
        wide = 0 if case["weight"] == "none" else SIZE[case["weight"]] * cols
        moved = 2 * n * size + 8 * rows + 2 * wide
        if case["train"]:
            moved += 3 * n * size + 8 * rows + 3 * wide      # x, dy read, dx written once more; w; dw, db
        return {"bytes": moved, "flops": n * (8 + (14 if case["train"] else 0))}
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * n * size + 4 * case["tokens"] * len(_numbers(case["axes"])), "flops": 3 * n}
    q_lens, k_lens, prefix = _numbers(case["q_lens"]), _numbers(case["k_lens"]), _numbers(case["prefix"])
    pairs = 0
    for n, (a, b) in enumerate(zip(q_lens, k_lens)):
        if not case["causal"]:
            pairs += a * b
        else:
            p = prefix[n] if prefix else 0
            pairs += sum(min(b, max(0, p, i + b - a + 1)) for i in range(a))
    q_bytes = sum(q_lens) * case["heads"] * case["dim"] * size
    k_bytes = sum(k_lens) * case["kv_heads"] * case["dim"] * size
    lse = 4 * sum(q_lens) * case["heads"]
    moved, flops = 2 * q_bytes + 2 * k_bytes + lse, 4 * case["dim"] * case["heads"] * pairs
    if case["train"]:
        moved += 4 * q_bytes + 4 * k_bytes + lse             # q, k, v, out, dout, lse read; dq, dk, dv written
        flops += 10 * case["dim"] * case["heads"] * pairs
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = (var + EPS).rsqrt()
        w = s["w"].double() if "w" in s else torch.ones(case["cols"], dtype=torch.float64, device="cuda")
        b = s["b"].double() if "b" in s else torch.zeros_like(w)
        result = {"y": (x - mean) * rstd * w + b, "mean": mean[:, 0], "rstd": rstd[:, 0]}
        if case["train"]:
            # the derivative written out: d y_c / d x_e = w_c rstd (1[c = e] - 1/C - hat_c hat_e / C)
            dy, hat = s["dy"].double(), (x - mean) * rstd
            inner = dy * w
            result["dx"] = rstd * (inner - (inner.sum(1, keepdim=True) + hat * (inner * hat).sum(1, keepdim=True))
                                   / case["cols"])
            if "w" in s:
                result["dw"], result["db"] = torch.einsum("rc,rc->c", dy, hat), dy.sum(0)
        return result
    if case["op"] == "rope":
        turn = []
        for n, width in enumerate(_numbers(case["axes"])):
            for i in range(width // 2):
                turn.append(s["positions"][:, n].double() * case["theta"] ** (-2.0 * i / width))
        angle = torch.stack(turn, dim=1)[:, None, :]
        unit = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
        result = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            r = 2 * len(turn)
            first, second = ((slice(0, r, 2), slice(1, r, 2)) if case["interleaved"]
                             else (slice(0, r // 2), slice(r // 2, r)))
            z = torch.complex(x[..., first], x[..., second]) * unit
            y[..., first], y[..., second] = z.real, z.imag
            result[name] = y
        return result
    q_lens, k_lens, prefix = _numbers(case["q_lens"]), _numbers(case["k_lens"]), _numbers(case["prefix"])
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    r = {"out": torch.zeros_like(s["q"], dtype=torch.float64),
         "lse": torch.full((h, sum(q_lens)), -math.inf, dtype=torch.float64, device="cuda")}
    if case["train"]:
        r |= {"d" + n: torch.zeros_like(s[n], dtype=torch.float64) for n in "qkv"}
    i0 = j0 = 0
    for n, (a, b) in enumerate(zip(q_lens, k_lens)):
        rows, cols = slice(i0, i0 + a), slice(j0, j0 + b)
        i0, j0 = i0 + a, j0 + b
        if a == 0 or b == 0:
            continue
        gap = torch.arange(b, device="cuda")[None, :] - (torch.arange(a, device="cuda")[:, None] + (b - a))
        hidden = torch.zeros_like(gap, dtype=torch.bool)
        if case["causal"]:
            hidden = gap > 0
            if prefix:
                hidden[:, :prefix[n]] = False
        for head in range(h):
            q, k, v = s["q"][rows, head].double(), s["k"][cols, head * g // h].double(), s["v"][cols, head * g // h].double()
            raw = q @ k.T / d ** 0.5
            z = raw if not case["cap"] else case["cap"] * torch.tanh(raw / case["cap"])
            if case["bias"]:
                z = z - s["slopes"][head].double() * gap.abs()
            z = z.masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(z, dim=1)
            p = torch.where(hidden, 0.0, torch.exp(z - lse[:, None]))
            r["out"][rows, head], r["lse"][head, rows] = p @ v, lse
            if case["train"]:
                do = s["dout"][rows, head].double()
                dz = p * (do @ v.T - (do * (p @ v)).sum(1, keepdim=True))
                if case["cap"]:
                    dz = dz * (1 - torch.tanh(raw / case["cap"]) ** 2)
                r["dq"][rows, head] = dz @ k / d ** 0.5
                r["dk"][cols, head * g // h] += dz.T @ q / d ** 0.5
                r["dv"][cols, head * g // h] += p.T @ do
    return r
