"""A transformer block over packed images and their texts, in training and for
single new tokens, with the package's operators.

The block is the one the residual-gate update belongs to:

    x + gate * (attention(rope(norm(q)), rope(norm(k)), v) W_o),  q, k, v = norm(x) W_qkv

over documents (an image's tokens behind its text's) that lie one after the
other along the token axis, each token with four positions (image, row, column,
text).  ``PackedBlock.forward`` and ``.backward`` show which results of the
forward calls the backward calls take; ``PackedBlock.decode`` adds one token to
every document beside a cache.  Matrix products are torch's.

    PYTHONPATH=. python examples/packed_image_block.py
"""
import torch

import channels_last_groupnorm_gb300 as gn

AXES, THETA, EPS = (32, 32, 32, 32), 2000.0, 1e-6


class PackedBlock:
    """Weights in bf16 (fp32 for the head norms): w_qkv [C, (H + 2 Hk) D], w_o [H D, C]."""

    def __init__(self, channels, heads, kv_heads, dim=128, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.w_qkv = (rand(channels, (heads + 2 * kv_heads) * dim) / channels ** 0.5).bfloat16()
        self.w_o = (rand(heads * dim, channels) / (heads * dim) ** 0.5).bfloat16()
        self.q_norm, self.k_norm = rand(dim) * 0.1 + 1.0, rand(dim) * 0.1 + 1.0
        self.gate = (rand(channels) * 0.5).bfloat16()

    def project(self, x, positions):
        """(what attention takes, what the backward pass needs)."""
        h, hk, d = self.heads, self.kv_heads, self.dim
        y, mean, rstd = gn.layer_norm(x, eps=EPS)
        qkv = (y @ self.w_qkv).view(x.shape[0], h + 2 * hk, d)
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        qn, q_mean, q_rstd = gn.layer_norm(q, self.q_norm, eps=EPS)
        kn, k_mean, k_rstd = gn.layer_norm(k, self.k_norm, eps=EPS)
        qr, kr = gn.rope_nd(qn, kn, positions, AXES, theta=THETA, out=(qn, kn))
        return qr, kr, v, (x, mean, rstd, y, q, q_mean, q_rstd, k, k_mean, k_rstd)

    def forward(self, x, positions, ends):
        """x [T, C] bf16, positions [T, 4] int32, ends int32 [documents + 1]."""
        q, k, v, saved = self.project(x, positions)
        out, lse = gn.attention_packed(q, k, v, ends, ends)
        update = out.flatten(1) @ self.w_o
        return gn.residual_gate_add(x, update, self.gate), (saved, q, k, v, out, lse, update, positions, ends)

    def backward(self, dz, kept):
        """The gradients of x and of every weight."""
        (x, mean, rstd, y, q0, q_mean, q_rstd, k0, k_mean, k_rstd), q, k, v, out, lse, update, positions, ends = kept
        d_update = dz * self.gate
        d_out = (d_update @ self.w_o.T).view_as(out)
        dq, dk, dv = gn.attention_packed_backward(d_out, q, k, v, out, lse, ends, ends)
        dq, dk = gn.rope_nd(dq, dk, positions, AXES, theta=THETA, inverse=True, out=(dq, dk))
        dq, d_q_norm, _ = gn.layer_norm_backward(dq, q0, q_mean, q_rstd, self.q_norm)
        dk, d_k_norm, _ = gn.layer_norm_backward(dk, k0, k_mean, k_rstd, self.k_norm)
        d_qkv = torch.cat([dq, dk, dv], dim=1).flatten(1)
        dx, _, _ = gn.layer_norm_backward(d_qkv @ self.w_qkv.T, x, mean, rstd)
        return dict(x=dz + dx, w_qkv=y.T @ d_qkv, w_o=out.flatten(1).T @ d_update, q_norm=d_q_norm, k_norm=d_k_norm,
                    gate=(dz.float() * update.float()).sum(0))

    def decode(self, x, positions, k_cache, v_cache, cache_ends):
        """One new token for each document: x [documents, C] beside caches of
        packed keys and values whose last one of each document is the token's
        own (written here)."""
        q, k, v, _ = self.project(x, positions)
        last = cache_ends[1:].long() - 1
        k_cache[last], v_cache[last] = k, v
        ends = torch.arange(x.shape[0] + 1, dtype=torch.int32, device=x.device)
        out, _ = gn.attention_packed(q, k_cache, v_cache, ends, cache_ends, causal=True)
        return gn.residual_gate_add(x, out.flatten(1) @ self.w_o, self.gate)


def packed_images(lens, texts, device="cuda"):
    """(ends, positions) of documents of `lens` tokens, the first `texts[n]` of them text."""
    ends = torch.tensor([0] + list(lens), device=device).cumsum(0).to(torch.int32)
    rows = []
    for n, (length, text) in enumerate(zip(lens, texts)):
        i = torch.arange(length, device=device)
        image = (i - text).clamp(min=0)
        side = max(1, int((length - text) ** 0.5))
        rows.append(torch.stack([torch.full_like(i, n), image // side, image % side, i.clamp(max=text)], dim=1))
    return ends, torch.cat(rows).to(torch.int32)


def main():
    block = PackedBlock(channels=1536, heads=12, kv_heads=4)
    ends, positions = packed_images([2048 + 128, 576 + 64, 1024 + 300], [128, 64, 300])
    x = torch.randn(int(ends[-1]), 1536, device="cuda").bfloat16()
    z, kept = block.forward(x, positions, ends)
    grads = block.backward(torch.randn_like(z), kept)
    print("trained on", tuple(z.shape), {n: tuple(g.shape) for n, g in grads.items()})
    caches = torch.zeros(2, int(ends[-1]), 4, 128, dtype=torch.bfloat16, device="cuda")
    caches[0], caches[1] = kept[2], kept[3]
    last = ends[1:].long() - 1
    new = block.decode(x[last], positions[last], caches[0], caches[1], ends)
    off = (new.float() - z[last].float()).norm() / z[last].float().norm()
    print("the last tokens again, one by one: off by", float(off))


if __name__ == "__main__":
    main()
