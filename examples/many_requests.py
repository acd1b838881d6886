"""A batch of requests on one quantized base model: they share a long prompt,
each has an adapter of its own, and their next tokens are scored.  One attention
layer and the vocabulary's product, served token by token; then a step of tuning
through the scores' gradient.

    python examples/many_requests.py
"""
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_step import AttentionLayer, mx  # noqa: E402


class SharedPromptLayer(AttentionLayer):
    """An attention layer whose requests share a prompt and name an adapter for
    the query, key and value projection, with the product that follows."""

    def __init__(self, hidden, vocab, requests, rank, adapters, seed=0, **kw):
        super().__init__(hidden, seed=seed, max_batch=requests, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        n = (self.heads + 2 * self.kv_heads) * self.dim
        self.adapters = mx.Adapters((r(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16),
                                    (r(adapters, n, rank) * 0.05).to(torch.bfloat16), torch.full((adapters,), 2.0, device="cuda"))
        self.w_vocab, _, _ = mx.mx_quantize(self.fmt, (r(vocab, hidden) * hidden ** -0.5).to(torch.bfloat16))

    def heads_of(self, x, ids, positions):
        """Queries, keys and values of tokens x (tokens x hidden) with their adapters."""
        t, h, k = x.shape[0], self.heads, self.kv_heads
        qkv = mx.mx_matvec(self.fmt, self.w_qkv, x, out_dtype=torch.float32)
        qkv = mx.mx_lora(x, self.adapters, ids, qkv, out_dtype=x.dtype).view(t, h + 2 * k, self.dim)
        q, key, value = qkv[:, :h], qkv[:, h:h + k], qkv[:, h + k:]
        mx.mx_qk_rope(q, key, self.cos, self.sin, positions, self.q_norm, self.k_norm, q_out=q, k_out=key)
        return q, key, value

    def prompt(self, x, prefix):
        """Writes the shared prompt's keys and values (no adapter) to the pages `prefix`."""
        t = torch.arange(x.shape[0], device=x.device)
        page = self.cache.page_size
        slots = prefix[t // page].long() * page + t % page
        _, key, value = self.heads_of(x, torch.full_like(t, -1, dtype=torch.int32), t.to(torch.int32))
        mx.mx_cache_write(self.cache, key, value, slots)
        return slots

    def logits(self, x, ids, positions, slots, prefix, prefix_length, page_table, lengths, workspace=None):
        """One new token of every request, behind the prompt and its own tokens."""
        q, key, value = self.heads_of(x, ids, positions)
        mx.mx_cache_write(self.cache, key, value, slots)
        o = mx.mx_attend_shared(q, self.cache, prefix, prefix_length, page_table, lengths, workspace=workspace)
        y = mx.mx_matvec(self.fmt, self.w_out, o.view(x.shape[0], self.heads * self.dim))
        return mx.mx_matvec(self.fmt, self.w_vocab, y, out_dtype=torch.float32)


class LogProbs(torch.autograd.Function):
    """mx_logprobs' logprob and entropy, and their gradient by the logits."""

    @staticmethod
    def forward(ctx, logits, targets):
        logprob, lse, entropy = mx.mx_logprobs(logits, targets)
        ctx.save_for_backward(logits, targets, lse, entropy)
        return logprob, entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, d_logprob, d_entropy):
        logits, targets, lse, entropy = ctx.saved_tensors
        dense = lambda t: None if t is None else t.float().contiguous()
        return mx.mx_logprobs_backward(dense(d_logprob), dense(d_entropy), logits, targets, lse, entropy), None


def main():
    dev, requests, prompt, steps, page = torch.device("cuda"), 6, 300, 20, 16
    layer = SharedPromptLayer(1024, 5000, requests, rank=16, adapters=4, q_heads=16, kv_heads=4, dim=64, pages=64, table_cols=40)
    prefix = torch.arange(-(-prompt // page), device=dev, dtype=torch.int32)
    length = torch.tensor([prompt], device=dev, dtype=torch.int32)
    slots = layer.prompt(torch.randn(prompt, 1024, device=dev).to(torch.bfloat16), prefix)
    k, _ = mx.mx_cache_read(layer.cache, slots)
    print(f"prompt of {prompt} tokens cached, norm of its keys {k.float().norm().item():.1f}")
    # request b's own tokens lie on pages 20 + 2 b and 21 + 2 b
    table = (20 + torch.arange(2 * requests, device=dev, dtype=torch.int32)).view(requests, 2)
    ids = torch.tensor([0, 1, 2, 3, 0, -1], device=dev, dtype=torch.int32)
    for t in range(steps):
        x = torch.randn(requests, 1024, device=dev).to(torch.bfloat16)
        at = torch.full((requests,), t, device=dev, dtype=torch.int32)
        own = table[:, t // page].long() * page + t % page
        z = layer.logits(x, ids, prompt + at, own, prefix, length, table, at + 1)
    logprob, lse, entropy, tops, top_ids = mx.mx_logprobs(z, z.argmax(1), top=5)
    print(f"after {steps} tokens: entropy {entropy.mean().item():.3f}, likeliest {top_ids[:, 0].tolist()}, "
          f"log probabilities {[round(v, 2) for v in logprob.tolist()]}")
    z = z.detach().requires_grad_()
    lp, h = LogProbs.apply(z, top_ids[:, 1].contiguous())
    (-lp.sum() - 0.01 * h.sum()).backward()
    print(f"gradient norm {z.grad.norm().item():.3f}")


if __name__ == "__main__":
    main()
