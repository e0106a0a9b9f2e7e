"""Serving a transformer block from a paged cache in 8 bits with the package's
operators: prompts in chunks, then single new tokens, through the same step.

    total = x + residual,  q, k, v = rms_norm(total) W_qkv
    append rope(k), v to the cache;  update = attention(rope(q), cache) W_o

``CachedBlock.step`` takes the packed new tokens of all sequences; the update and
the residual stream (``total``) go to the next block's norm, which adds them.  Matrix
products are torch's.

    PYTHONPATH=. python examples/cached_block.py
"""
import torch

import channels_last_groupnorm_gb300 as gn

AXES, THETA, EPS = (128,), 10000.0, 1e-6


class PagedCache:
    """Pages for some sequences, handed out from a pool as they grow.  A head's tokens of a
    page lie next to each other."""

    def __init__(self, sequences, pages, kv_heads, dim=128, page_size=64, width=None, device="cuda"):
        self.page_size, self.free = page_size, list(range(pages))
        self.k_pages, self.v_pages = (
            torch.zeros(pages, kv_heads, page_size, dim, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn).transpose(1, 2)
            for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros(pages, kv_heads, device=device) for _ in range(2))
        self.rows = [[] for _ in range(sequences)]
        self.held = [0] * sequences
        self.table = torch.zeros(sequences, width or pages, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device=device)

    def grow(self, new):
        """Room for new[s] more tokens of every sequence; their ends among the packed ones."""
        for s, n in enumerate(new):
            self.held[s] += n
            while len(self.rows[s]) * self.page_size < self.held[s]:
                self.rows[s].append(self.free.pop())
            if self.rows[s]:
                self.table[s, :len(self.rows[s])] = torch.tensor(self.rows[s], dtype=torch.int32)
        self.lengths.copy_(torch.tensor(self.held, dtype=torch.int32))
        return torch.tensor([0] + list(new), device=self.table.device).cumsum(0).to(torch.int32)

    def args(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales, self.table, self.lengths


class CachedBlock:
    """Weights in bf16: w_qkv [C, (H + 2 Hk) D], w_o [H D, C], norm [C]."""

    def __init__(self, channels, heads, kv_heads, dim=128, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.w_qkv = (rand(channels, (heads + 2 * kv_heads) * dim) / channels ** 0.5).bfloat16()
        self.w_o = (rand(heads * dim, channels) / (heads * dim) ** 0.5).bfloat16()
        self.norm = (rand(channels) * 0.1 + 1.0).bfloat16()

    def step(self, x, residual, positions, cache, cu):
        """x and residual [T, C] bf16, positions [T, 1] int32, cu int32 [sequences + 1]:
        (update, total), the cache holding the new tokens."""
        h, hk = self.heads, self.kv_heads
        y, _, total, _ = gn.rms_norm(x, self.norm, residual=residual, eps=EPS)
        qkv = (y @ self.w_qkv).view(x.shape[0], h + 2 * hk, self.dim)
        q = gn.cache_append(qkv[:, h:h + hk], qkv[:, h + hk:], *cache.args(), cu, q=qkv[:, :h], positions=positions,
                            axes_dim=AXES, theta=THETA)
        out, _ = gn.attention_cached(q, *cache.args(), cu)
        return out.flatten(1) @ self.w_o, total


def places(held, new, device="cuda"):
    """The new tokens' positions, sequence by sequence."""
    return torch.cat([torch.arange(h - n, h) for h, n in zip(held, new)]).to(torch.int32).to(device)[:, None]


def main():
    block = CachedBlock(channels=1536, heads=12, kv_heads=4)
    cache = PagedCache(sequences=3, pages=80, kv_heads=4)
    for new in ([1000, 300, 41], [500, 0, 900], [1, 1, 1], [1, 1, 1]):
        cu = cache.grow(new)
        x, residual = torch.randn(2, sum(new), 1536, device="cuda").bfloat16()
        update, total = block.step(x, residual, places(cache.held, new), cache, cu)
        print("new", new, "held", cache.held, "update", tuple(update.shape), float(update.float().std()))


if __name__ == "__main__":
    main()
