"""One attention layer served token by token with quantized weights and a
quantized key-value cache: the product with the 4-bit projections, the norm and
rotation of the heads, the write to the paged cache, the attention over it, and
the output projection; then the same heads' norm and rotation in a training
step, through autograd.

    python examples/decode_step.py
"""
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_block_quantization_amd as mx  # noqa: E402


def rotation_tables(positions, rot_dim, device, base=10000.0):
    """cos and sin of every position's angles, fp32."""
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return a.cos().float().to(device), a.sin().float().to(device)


class AttentionLayer:
    """Weights in `fmt` (any format mx_matvec takes), a cache in `cache_fmt`
    (None: bf16), both laid out once."""

    def __init__(self, hidden, q_heads, kv_heads, dim, fmt=mx.MXFP4, cache_fmt=mx.MXFP8_E4M3, pages=64, page_size=16,
                 max_batch=16, table_cols=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        weight = lambda n, k: (torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(torch.bfloat16)
        self.heads, self.kv_heads, self.dim, self.fmt = q_heads, kv_heads, dim, fmt
        self.w_qkv, _, _ = mx.mx_quantize(fmt, weight((q_heads + 2 * kv_heads) * dim, hidden))
        self.w_out, _, _ = mx.mx_quantize(fmt, weight(hidden, q_heads * dim))
        norm = lambda: (1 + 0.1 * torch.randn(dim, generator=g, device=device)).to(torch.bfloat16)
        self.q_norm, self.k_norm = norm(), norm()
        self.cos, self.sin = rotation_tables(page_size * table_cols, dim, device)
        self.cache = mx.alloc_kv_cache(cache_fmt, pages, page_size, kv_heads, dim, device)
        self.workspace = mx.alloc_attend_workspace(self.cache, max_batch, q_heads, table_cols)

    def step(self, x, positions, slots, page_table, lengths):
        """x: batch x hidden, one new token per sequence at positions[b], whose
        key and value go to slots[b]; lengths[b] counts it."""
        b, h, k = x.shape[0], self.heads, self.kv_heads
        qkv = mx.mx_matvec(self.fmt, self.w_qkv, x).view(b, h + 2 * k, self.dim)
        q, key, value = qkv[:, :h], qkv[:, h:h + k], qkv[:, h + k:]
        mx.mx_qk_rope(q, key, self.cos, self.sin, positions, self.q_norm, self.k_norm, q_out=q, k_out=key)
        mx.mx_cache_write(self.cache, key, value, slots)
        o = mx.mx_attend(q, self.cache, page_table, lengths, workspace=self.workspace)
        return mx.mx_matvec(self.fmt, self.w_out, o.view(b, h * self.dim))


class QKRope(torch.autograd.Function):
    """mx_qk_rope and its gradient for training; k and either weight may be None."""

    @staticmethod
    def forward(ctx, q, k, cos, sin, positions, q_weight, k_weight, eps):
        ctx.save_for_backward(q, k, cos, sin, positions, q_weight, k_weight)
        ctx.eps = eps
        return mx.mx_qk_rope(q, k, cos, sin, positions, q_weight, k_weight, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy_q, dy_k):
        q, k, cos, sin, positions, qw, kw = ctx.saved_tensors
        dense = lambda t: None if t is None else t.contiguous()
        dq, dk, dqw, dkw = mx.mx_qk_rope_backward(dense(dy_q), dense(dy_k), q, k, cos, sin, positions, qw, kw, ctx.eps)
        like = lambda g, w: None if w is None else g.to(w.dtype)
        return dq, dk, None, None, None, like(dqw, qw), like(dkw, kw), None


def main():
    hidden, batch, steps, page = 1024, 3, 40, 16
    layer = AttentionLayer(hidden, q_heads=16, kv_heads=4, dim=64)
    dev = torch.device("cuda")
    # sequence b owns pages b * 4 .. b * 4 + 3
    table = torch.arange(batch * 4, device=dev, dtype=torch.int32).view(batch, 4)
    table = torch.nn.functional.pad(table, (0, 12), value=-1)
    for t in range(steps):
        x = torch.randn(batch, hidden, device=dev).to(torch.bfloat16)
        at = torch.full((batch,), t, device=dev, dtype=torch.int32)
        slots = table[:, t // page].long() * page + t % page
        y = layer.step(x, at, slots, table, at + 1)
    print(f"{steps} tokens for {batch} sequences, last output norm {y.float().norm().item():.3f}")
    q, k = (torch.randn(50, h, 64, device=dev, dtype=torch.bfloat16, requires_grad=True) for h in (16, 4))
    qw, kw = (torch.ones(64, device=dev, dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    yq, yk = QKRope.apply(q, k, layer.cos, layer.sin, torch.arange(50, device=dev, dtype=torch.int32), qw, kw, 1e-6)
    (yq.float().square().sum() + yk.float().sum()).backward()
    print(f"gradient norms: q {q.grad.float().norm().item():.3f}, k {k.grad.float().norm().item():.3f}, "
          f"k weight {kw.grad.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
