"""The operators of serving from an 8-bit cache of keys and values, as they are measured.

Three operators that stand next to the package's layer norm, rotary positions
and packed attention:

  rms         y = t rstd w of t = x + residual, rstd = 1 / sqrt(mean(t^2) + eps),
              in the input's type or as e4m3 with a scale for each row, and its
              backward pass with the reduction of the weight's gradient;
  append      new tokens' keys (turned by the rotary positions on the way) and
              values into a paged cache of e4m3 with a scale for each page and
              head, and the query heads turned in the same call;
  attention   of new tokens over such a cache: each query sees its sequence's
              tokens up to its own position, scores optionally capped by a tanh
              and biased by the distance, with grouped key / value heads.

A page's scale is the power of two with which its largest magnitude just fits
under 448; a page that is filled further keeps its scale or, where a new token
does not fit, has what it holds rounded to the larger one.

With ``own`` false, ``run`` evaluates the formulas with elementary torch
operations; with ``own`` true it calls the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
LEAST = -100          # exponent of the smallest scale of a page


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
CACHES = "8000,17,3501,1,6007,129,4096,777,2048,5555,64,7013,333,1000,4999,2500,1,6500,88,3030,7777,15,450,5120"


def listed():
    return [
        # the norm ahead of a projection in 8 bits, one new token with the update before it added
        dict(name="rms_one_token", op="rms", tokens=1, heads=0, cols=6144, type="bf16", weight="bf16", residual=True,
             out="e4m3", train=False),
        # the same over the 4096 image and 512 text tokens of a 1024 x 1024 image
        dict(name="rms_image_e4m3", op="rms", tokens=4608, heads=0, cols=6144, type="bf16", weight="bf16", residual=True,
             out="e4m3", train=False),
        # a training step of that norm, the residual stream's own gradient added on the way back
        dict(name="rms_train_image", op="rms", tokens=4608, heads=0, cols=6144, type="bf16", weight="fp32", residual=True,
             out="same", train=True),
        # the norm of every query head of a fused projection ahead of the rotation: very many short rows
        dict(name="rms_train_heads", op="rms", tokens=4608, heads=24, cols=128, type="fp16", weight="fp16", residual=False,
             out="same", train=True),
        # odd width and row count in full precision
        dict(name="rms_train_odd", op="rms", tokens=3001, heads=0, cols=1003, type="fp32", weight="fp32", residual=True,
             out="same", train=True),
        # one new token for each of many sequences: pages that are filled to different heights
        dict(name="append_one_token", op="append", new="1," * 23 + "1", lens=CACHES, heads=32, kv_heads=8, dim=128, page=64,
             axes="32,32,32,32", theta=2000.0, interleaved=True, type="bf16"),
        # the prompts of several images with their texts, one of them behind tokens that are there already
        dict(name="append_images", op="append", new="4608,1536,2111,300", lens="4608,1536,2111,700", heads=24, kv_heads=24,
             dim=128, page=64, axes="32,32,32,32", theta=2000.0, interleaved=True, type="bf16"),
        # a chunk of video tokens behind others, halves paired, an unrotated rest, large pages
        dict(name="append_video", op="append", new="7003,1001", lens="30011,1500", heads=12, kv_heads=3, dim=112, page=128,
             axes="24,36,36", theta=10000.0, interleaved=False, type="fp16"),
        # one new token for each of many sequences, grouped heads
        dict(name="cached_one_token", op="attn", new="1," * 23 + "1", lens=CACHES, heads=32, kv_heads=8, dim=128, page=64,
             cap=0.0, bias=False, type="bf16"),
        # four proposed tokens each for a few sequences, small pages, capped scores
        dict(name="cached_four_tokens", op="attn", new="4,4,4,4,4,4,4", lens="1001,16384,4,250,9000,3333,40", heads=32,
             kv_heads=4, dim=64, page=16, cap=50.0, bias=False, type="fp16"),
        # one token far into a single long sequence
        dict(name="cached_far_token", op="attn", new="1", lens="131072", heads=32, kv_heads=8, dim=128, page=128, cap=0.0,
             bias=False, type="bf16"),
        # a chunk of a long prompt and the whole of a short one
        dict(name="cached_chunk", op="attn", new="2048,1111", lens="16384,1111", heads=32, kv_heads=8, dim=128, page=64,
             cap=0.0, bias=False, type="bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rms", "append", "attn", "attn"])
    kind = rng.choice(["bf16", "fp16"])
    if op == "rms":
        heads = rng.choice([0, 0, 4, 12])
        cols = rng.choice([64, 72, 96, 128]) if heads else _log(rng, 32, 12288)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        kind = rng.choice(["bf16", "fp16", "fp32"])
        train = rng.random() < 0.5
        tokens = _log(rng, 1, min(100000, 28_000_000 // (cols * max(1, heads))))
        return dict(op="rms", tokens=tokens, heads=heads, cols=cols, type=kind, weight=rng.choice(["none", "fp32", kind]),
                    residual=not heads and rng.random() < 0.7, out="same" if train else rng.choice(["same", "e4m3", "e4m3"]),
                    train=train)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 8])
    page = rng.choice([16, 32, 64, 64, 128])
    count = _log(rng, 1, 24)
    if op == "append":
        axes = rng.choice(["32,32,32,32", "16,56,56", "24,36,36", "64", "16,24,24", "80"])
        width = sum(int(a) for a in axes.split(","))
        dim = min(128, (width + rng.choice([0, 0, 16]) + 15) // 16 * 16)
        most = min(8000, 40_000_000 // (dim * (heads + 2 * kv_heads))) // count
        new = [1] * count if rng.random() < 0.3 else [_log(rng, 1, max(1, most)) for _ in range(count)]
        lens = [n + rng.choice([0, rng.randint(0, 2 * page), rng.randint(0, 4000)]) for n in new]
        return dict(op="append", new=_text(new), lens=_text(lens), heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    axes=axes, theta=rng.choice([2000.0, 10000.0, 1000000.0]), interleaved=rng.random() < 0.5,
                    type=rng.choice(["bf16", "fp16", "fp32"]))
    dim = rng.choice([64, 64, 128, 128, 96, 80])
    common = dict(op="attn", heads=heads, kv_heads=kv_heads, dim=dim, page=page, cap=rng.choice([0.0, 0.0, 0.0, 30.0]),
                  bias=rng.random() < 0.2, type=kind)
    if rng.random() < 0.6:                       # new tokens: one for each sequence, or a few
        new = [rng.choice([1, 1, 2, 3, 5])] * count
        return dict(new=_text(new), lens=_text([_log(rng, new[0], 8192 if count > 2 else 32768) for _ in new]), **common)
    count = min(count, 6)
    new = [_log(rng, 1, 1200 // count) for _ in range(count)]
    return dict(new=_text(new), lens=_text([n + rng.choice([0, rng.randint(0, 6000)]) for n in new]), **common)


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
    if case["op"] == "rms":
        tokens, heads, cols = case["tokens"], case["heads"], case["cols"]
        if heads:                                             # some heads of a fused projection
            state["x"] = normal(tokens, heads + 2, cols, scale=2.0)[:, :heads]
        else:
            # channels of a residual stream: a few of them large; the update is small beside it
            size = 1.0 + 0.2 * normal(cols, to=torch.float32)
            size[:: max(1, cols // 3)] *= 20.0
            state["x"] = (normal(tokens, cols, to=torch.float32) * (0.5 if case["residual"] else size)).to(kind)
            if case["residual"]:
                state["stream"] = (normal(tokens, cols, to=torch.float32) * size).to(kind)
        if case["weight"] != "none":
            state["w"] = normal(cols, scale=0.2, to=torch.float32).add_(1.0).to(TYPES[case["weight"]])
        if case["train"]:
            state["dy"] = normal(*state["x"].shape)
            if case["residual"]:
                state["dtotal"] = normal(*state["x"].shape)
        return state
    new, lens = _numbers(case["new"]), _numbers(case["lens"])
    h, g, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    tokens = sum(new)
    # every sequence has the pages that it needs, from anywhere in a pool with some to spare
    wants = [(n + page - 1) // page for n in lens]
    width, pages = max(wants), sum(wants) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    ends = torch.tensor([0] + wants, device="cuda").cumsum(0)
    column = torch.arange(width, device="cuda")[None, :]
    state["table"] = torch.where(column < (ends[1:] - ends[:-1])[:, None],
                                 order[(ends[:-1, None] + column).clamp(max=pages - 1)], 0)
    state["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    state["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    for name in ("k", "v"):
        # values of one head lie next to each other within a page
        values = normal(pages, g, page, d, scale=1.4 if name == "k" else 1.0, to=torch.float32)
        values *= torch.exp2(normal(pages, g, 1, 1, to=torch.float32))
        scale = _scale_of(values.abs().amax(dim=(2, 3)))
        state[name + "_pages"] = (values / scale[:, :, None, None]).to(E4M3).transpose(1, 2)
        state[name + "_scales"] = scale
    if case["op"] == "append":
        qkv = normal(tokens, h + 2 * g, d, scale=1.4)         # the fused projection of a block
        state["q"], state["k"], state["v"] = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        token = torch.arange(tokens, device="cuda") + int(torch.randint(0, 1000, (), generator=gen, device="cuda"))
        parts = [token // 4096, token // 64 % 64, token % 64, token]
        state["positions"] = torch.stack(parts[:len(_numbers(case["axes"]))], dim=1).to(torch.int32)
    else:
        state["q"] = normal(tokens, h, d, scale=1.4)
        state["slopes"] = (torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda", dtype=torch.float32) / h)
                           if case["bias"] else None)
        if len(set(new)) == 1:                                # equally many for each sequence: nothing to tell
            state["cu"] = None
    return state


def _scale_of(amax):
    """The least power of two of which 448 times is no less, 2^LEAST at least."""
    fraction, exponent = torch.frexp(amax)
    exponent = (exponent - 9 + (fraction > 0.875).int()).clamp(min=LEAST)
    return torch.where(torch.isfinite(amax), torch.ldexp(torch.ones_like(amax), exponent), math.nan)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"rms": _plain_rms, "append": _plain_append, "attn": _plain_attn}[state["op"]](state)


def _run_own(s):
    import channels_last_groupnorm_gb300 as gn

    if s["op"] == "rms":
        y, scales, total, rstd = gn.rms_norm(s["x"], s.get("w"), residual=s.get("stream"), eps=EPS,
                                             quantize=s["out"] == "e4m3")
        result = _some(y=y, scales=scales, total=total if s["residual"] else None, rstd=rstd)
        if s["train"]:
            result["dx"], dw = gn.rms_norm_backward(s["dy"], total, rstd, s.get("w"), dtotal=s.get("dtotal"))
            result |= _some(dw=dw)
        return result
    if s["op"] == "append":
        q = gn.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                            s["lengths"], s["cu"], q=s["q"], positions=s["positions"], axes_dim=_numbers(s["axes"]),
                            theta=s["theta"], interleaved=s["interleaved"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "k_scales": s["k_scales"],
                "v_scales": s["v_scales"]}
    out, lse = gn.attention_cached(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                                   s["lengths"], s["cu"], slopes=s["slopes"], cap=s["cap"])
    return {"out": out, "lse": lse}


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _plain_rms(s):
    kind = s["x"].dtype
    total = s["x"]
    if s["residual"]:
        total = (s["x"].float() + s["stream"].float()).to(kind)
    t = total.float()
    rstd = 1.0 / torch.sqrt((t * t).mean(dim=-1) + EPS)
    hat = t * rstd[..., None]
    w = s["w"].float() if "w" in s else torch.ones(s["cols"], device="cuda")
    y, scales = hat * w, None
    if s["out"] == "e4m3":
        most = y.abs().amax(dim=-1)
        scales = most / 448.0
        y = (y * (448.0 / most)[..., None]).clamp(-448.0, 448.0).to(E4M3)
    else:
        y = y.to(kind)
    result = _some(y=y, scales=scales, total=total if s["residual"] else None, rstd=rstd)
    if s["train"]:
        dy = s["dy"].float()
        grad = dy * w
        dx = rstd[..., None] * (grad - hat * (grad * hat).mean(dim=-1, keepdim=True))
        if s["residual"]:
            dx = dx + s["dtotal"].float()
        result["dx"] = dx.to(kind)
        if "w" in s:
            result["dw"] = (dy * hat).flatten(0, -2).sum(dim=0).to(s["w"].dtype)
    return result


def _turned(x, s):
    """x in fp32, turned by its tokens' positions."""
    axes = _numbers(s["axes"])
    pairs = torch.tensor([a // 2 for a in axes], device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(axes), device="cuda"), pairs, output_size=sum(axes) // 2)
    place = torch.arange(axis.numel(), device="cuda") - (pairs.cumsum(0) - pairs)[axis]
    # angles in 64 bits: far positions lose their phase in 32
    rate = torch.exp(-math.log(s["theta"]) * place.double() / pairs[axis].double())
    angle = (s["positions"].double()[:, axis] * rate)[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    half = cos.shape[-1]
    f = x.float()
    r = f[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], dim=-1).flatten(-2) if s["interleaved"] else torch.cat([u, v], dim=-1)
    return torch.cat([y, f[..., 2 * half:]], dim=-1)


def _plain_append(s):
    cu, lengths, table, page = s["cu"].long(), s["lengths"].long(), s["table"].long(), s["page"]
    token = torch.arange(s["k"].shape[0], device="cuda")
    seq = (token[:, None] >= cu[1:][None, :]).sum(dim=1)
    new = cu[1:] - cu[:-1]
    place = lengths[seq] - new[seq] + token - cu[seq]
    at, slot = table[seq, place // page], place % page
    # the pages that are filled further: each sequence's first one, where it does not begin in it
    begin = lengths - new
    old, there = table[torch.arange(new.numel(), device="cuda"), begin // page], begin % page
    for name, rows in (("k", _turned(s["k"], s)), ("v", s["v"].float())):
        pool, scales = s[name + "_pages"], s[name + "_scales"]
        most = torch.zeros_like(scales)
        most.scatter_reduce_(0, at[:, None].expand(-1, most.shape[1]), rows.abs().amax(dim=2), "amax")
        need = _scale_of(most)
        before = scales[old]
        scales[at] = need[at]
        scales[old] = torch.where((there > 0)[:, None], torch.maximum(before, need[old]), need[old])
        held = pool[old].float() * (before / scales[old])[:, None, :, None]
        kept = torch.arange(page, device="cuda")[None, :] < there[:, None]
        bytes_of = pool.view(torch.uint8)
        bytes_of[old] = torch.where(kept[:, :, None, None], held.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8),
                                    bytes_of[old])
        bytes_of[at, slot] = (rows / scales[at][:, :, None]).to(E4M3).view(torch.uint8)
    return {"q": _turned(s["q"], s).to(s["q"].dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"],
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_attn(s):
    heads, g, d, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    lengths, table = s["lengths"].long(), s["table"].long()
    count, tokens = lengths.numel(), s["q"].shape[0]
    most = max(_numbers(s["new"]))
    if s["cu"] is None:
        cu = torch.arange(count + 1, device="cuda") * (tokens // count)
    else:
        cu = s["cu"].long()
    new = cu[1:] - cu[:-1]
    # every sequence's queries and its whole table of pages, padded to the longest
    i = torch.arange(most, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    q = s["q"][at].float().view(count, most, g, heads // g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = (((s[n + "_pages"][table].float() * s[n + "_scales"][table][:, :, None, :, None])
             .flatten(1, 2).transpose(1, 2)) for n in "kv")                    # [sequences, g, keys, d]
    j = torch.arange(k.shape[2], device="cuda")
    place = lengths[:, None] - new[:, None] + i                                # of each query
    seen = (j <= place[:, :, None]) & (i < new[:, None])[:, :, None]           # [sequences, queries, keys]
    scores = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (heads // g, most)) * (1.0 / math.sqrt(d))
    if s["cap"]:
        scores = torch.tanh(scores / s["cap"]) * s["cap"]
    if s["slopes"] is not None:
        away = (place[:, :, None] - j).abs().float()
        scores = scores - s["slopes"].view(1, g, heads // g, 1, 1) * away[:, None, None]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    del scores
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]                                     # [sequences, g, heads / g, queries]
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (heads // g, most))
    # back to the packed order
    token = torch.arange(tokens, device="cuda")
    seq = (token[:, None] >= cu[1:][None, :]).sum(dim=1)
    row = token - cu[seq]
    out = out.permute(0, 3, 1, 2, 4)[seq, row].flatten(1, 2)
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[seq, row].flatten(1, 2).T}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "rms":
        rows, cols = case["tokens"] * max(1, case["heads"]), case["cols"]
        n, wide = rows * cols, 0 if case["weight"] == "none" else SIZE[case["weight"]] * cols
        moved = n * size + 4 * rows + wide + (n + 4 * rows if case["out"] == "e4m3" else n * size)
        if case["residual"]:
            moved += 2 * n * size
        if case["train"]:
            moved += 3 * n * size + 4 * rows + 2 * wide + (n * size if case["residual"] else 0)
        return {"bytes": moved, "flops": n * (5 + (10 if case["train"] else 0))}
    new, lens = _numbers(case["new"]), _numbers(case["lens"])
    h, g, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        touched = sum((b - 1) // page - (b - a) // page + 1 for a, b in zip(new, lens))
        moved = sum(new) * ((2 * h + 2 * g) * d * size + 2 * g * d + 4 * len(_numbers(case["axes"])))
        return {"bytes": moved + 2 * 4 * g * (touched + len(new)), "flops": sum(new) * d * (3 * h + 6 * g)}
    pairs = sum(sum(range(b - a + 1, b + 1)) for a, b in zip(new, lens))
    held = sum(lens) * g * d * 2 + sum((b + page - 1) // page for b in lens) * (g * 2 * 4 + 4)
    return {"bytes": sum(new) * h * (2 * d * size + 4) + held, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _to_e4m3(x):
    """The nearest number of four bits of precision, 2^-9 the smallest step, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rms":
        total = s["x"]
        if case["residual"]:
            total = (s["x"].double() + s["stream"].double()).to(s["x"].dtype)   # what is stored and normed
        t = total.double()
        rstd = (t.square().sum(dim=-1) / case["cols"] + EPS).rsqrt()
        w = s["w"].double() if "w" in s else torch.ones(case["cols"], dtype=torch.float64, device="cuda")
        y = t * rstd.unsqueeze(-1) * w
        r = {"y": y}
        if case["out"] == "e4m3":
            r["scales"] = y.abs().max(dim=-1).values / 448
            r["y"] = _to_e4m3(y / r["scales"].unsqueeze(-1))
        if case["residual"]:
            r["total"] = total.double()
        r["rstd"] = rstd
        if case["train"]:
            # the derivative written out: d y_c / d t_e = w_c rstd (1[c = e] - t_c t_e rstd^2 / C)
            dy = s["dy"].double()
            along = torch.einsum("...c,...c->...", dy * w, t) / case["cols"]
            r["dx"] = rstd.unsqueeze(-1) * dy * w - t * (along * rstd ** 3).unsqueeze(-1)
            if case["residual"]:
                r["dx"] += s["dtotal"].double()
            if "w" in s:
                r["dw"] = (dy * t * rstd.unsqueeze(-1)).reshape(-1, case["cols"]).sum(0)
        return r
    new, lens = _numbers(case["new"]), _numbers(case["lens"])
    h, g, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    starts = [sum(new[:n]) for n in range(len(new))]
    if case["op"] == "append":
        turn = []
        for n, width in enumerate(_numbers(case["axes"])):
            for i in range(width // 2):
                turn.append(s["positions"][:, n].double() * case["theta"] ** (-2.0 * i / width))
        angle = torch.stack(turn, dim=1)[:, None, :]
        unit = torch.polar(torch.ones_like(angle), angle)
        count = 2 * len(turn)
        first, second = ((slice(0, count, 2), slice(1, count, 2)) if case["interleaved"]
                         else (slice(0, count // 2), slice(count // 2, count)))

        def turned(x):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * unit
            y[..., first], y[..., second] = z.real, z.imag
            return y

        r = {"q": turned(s["q"])}
        rows = {"k": turned(s["k"]), "v": s["v"].double()}
        for name in "kv":
            r[name + "_pages"] = s[name + "_pages"].double()
            r[name + "_scales"] = s[name + "_scales"].double()
        tables = s["table"].tolist()
        for name in "kv":
            pool, scales = r[name + "_pages"], r[name + "_scales"]
            for n, (count_new, length) in enumerate(zip(new, lens)):
                for p in range((length - count_new) // page, (length - 1) // page + 1):
                    a, b = max(length - count_new, p * page), min(length, (p + 1) * page)
                    at = starts[n] + a - (length - count_new)
                    x = rows[name][at:at + b - a]                             # [tokens, g, d]
                    room, was = pool[tables[n][p]], scales[tables[n][p]]
                    # (a quotient that is a power of two may have a logarithm a rounding above its exponent)
                    want = torch.log2(x.abs().amax(dim=(0, 2)) / 448) - 1e-12
                    want = torch.exp2(torch.ceil(want).clamp(min=LEAST))
                    now = torch.maximum(want, was) if a > p * page else want
                    low = a - p * page
                    room[:low] = _to_e4m3(room[:low] * (was / now)[:, None])
                    room[low:low + b - a] = _to_e4m3(x / now[:, None])
                    was.copy_(now)
        return {n: r[n] for n in ("q", "k_pages", "v_pages", "k_scales", "v_scales")}
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    lse = torch.full((h, sum(new)), -math.inf, dtype=torch.float64, device="cuda")
    for n, (count_new, length) in enumerate(zip(new, lens)):
        rows = slice(starts[n], starts[n] + count_new)
        used = s["table"][n, :(length + page - 1) // page].long()
        gap = (torch.arange(length, device="cuda")[None, :]
               - torch.arange(length - count_new, length, device="cuda")[:, None])
        for head in range(h):
            kv = []
            for name in "kv":
                room = s[name + "_pages"][used][:, :, head * g // h].double()
                kv.append((room * s[name + "_scales"][used][:, head * g // h].double()[:, None, None]).flatten(0, 1)[:length])
            z = s["q"][rows, head].double() @ kv[0].T / d ** 0.5
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if case["bias"]:
                z = z - s["slopes"][head].double() * gap.abs()
            z = z.masked_fill(gap > 0, -math.inf)
            lse[head, rows] = torch.logsumexp(z, dim=1)
            out[rows, head] = torch.exp(z - lse[head, rows, None]) @ kv[1]
    return {"out": out, "lse": lse}
