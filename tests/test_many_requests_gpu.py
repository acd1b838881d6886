"""The calls that serve many requests, together: a batch behind a shared prompt
with adapters, served step by step, against the same sequences served one at a
time by the calls that were there before, and in a captured graph; the scores'
gradient through autograd; the example."""
import os
import subprocess
import sys

import pytest
import torch

import microscaling_block_quantization_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
from many_requests import LogProbs, SharedPromptLayer  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
PAGE, PROMPT, REQUESTS = 16, 100, 5


def setup(fmt, cache_fmt):
    layer = SharedPromptLayer(512, 1000, REQUESTS, rank=16, adapters=3, fmt=fmt, cache_fmt=cache_fmt, q_heads=8, kv_heads=2, dim=64,
                              pages=40, table_cols=20)
    g = torch.Generator(device="cuda").manual_seed(3)
    prefix = torch.randperm(20, generator=g, device="cuda")[:7].to(torch.int32)
    table = (20 + torch.randperm(20, generator=g, device="cuda")[:2 * REQUESTS]).to(torch.int32).view(REQUESTS, 2)
    ids = torch.tensor([2, 0, -1, 0, 1], device="cuda", dtype=torch.int32)
    return layer, prefix, table, ids, torch.randn(PROMPT, 512, generator=g, device="cuda").to(BF16), g


@pytest.mark.parametrize("fmt,cache_fmt", [(mx.MXFP4, mx.MXFP8_E4M3), (mx.Format(scale=mx.SCALE_NVFP4, block_cols=16), None),
                                           (mx.MXFP4, mx.MXFP4)])
def test_against_one_at_a_time(fmt, cache_fmt):
    layer, prefix, table, ids, x, g = setup(fmt, cache_fmt)
    layer.prompt(x, prefix)
    length = torch.tensor([PROMPT], device="cuda", dtype=torch.int32)
    for t in range(18):
        x = torch.randn(REQUESTS, 512, generator=g, device="cuda").to(BF16)
        at = torch.full((REQUESTS,), t, device="cuda", dtype=torch.int32)
        slots = table[:, t // PAGE].long() * PAGE + t % PAGE
        q, key, value = layer.heads_of(x, ids, PROMPT + at)
        mx.mx_cache_write(layer.cache, key, value, slots)
        o, lse = mx.mx_attend_shared(q, layer.cache, prefix, length, table, at + 1, lse=True)
        # the products and adapters of each token alone
        for b in range(REQUESTS):
            q1, k1, v1 = layer.heads_of(x[b:b + 1], ids[b:b + 1], (PROMPT + at)[b:b + 1])
            assert (q1[0].float() - q[b].float()).abs().max() <= 2.0 ** -7 * q[b].float().abs().max()
        # the prompt's tokens read back and written ahead of each request's own
        if t in (0, 17):
            tok = torch.arange(PROMPT, device="cuda")
            pk, pv = mx.mx_cache_read(layer.cache, prefix[tok // PAGE].long() * PAGE + tok % PAGE, out_dtype=torch.float32)
            for b in range(REQUESTS):
                mine = torch.arange(t + 1, device="cuda")
                ok, ov = mx.mx_cache_read(layer.cache, table[b, mine // PAGE].long() * PAGE + mine % PAGE, out_dtype=torch.float32)
                one = mx.alloc_kv_cache(cache_fmt, 12, PAGE, 2, 64)
                mx.mx_cache_write(one, torch.cat((pk, ok)), torch.cat((pv, ov)), torch.arange(PROMPT + t + 1, device="cuda"))
                w, l1 = mx.mx_attend(q[b:b + 1], one, torch.arange(12, device="cuda", dtype=torch.int32)[None],
                                     torch.tensor([PROMPT + t + 1], device="cuda", dtype=torch.int32), lse=True)
                assert (w[0].float() - o[b].float()).abs().max() <= 2.0 ** -7 * w.float().abs().max()
                assert (l1[0] - lse[b]).abs().max() < 1e-5


def test_graph_of_a_step():
    """The whole step captured once and replayed with other tokens, places and adapters."""
    layer, prefix, table, ids, x, g = setup(mx.MXFP4, mx.MXFP8_E4M3)
    layer.prompt(x, prefix)
    length = torch.tensor([PROMPT], device="cuda", dtype=torch.int32)
    x = torch.randn(REQUESTS, 512, device="cuda").to(BF16)
    at = torch.zeros(REQUESTS, device="cuda", dtype=torch.int32)
    slots = table[:, 0].long() * PAGE
    target = torch.zeros(REQUESTS, device="cuda", dtype=torch.int64)
    ws = mx.alloc_attend_shared_workspace(layer.cache, REQUESTS, 8, 7, 2)
    step = lambda: mx.mx_logprobs(layer.logits(x, ids, PROMPT + at, slots, prefix, length, table, at + 1, ws), target, top=5)
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step()
    for t in range(5):
        x.copy_(torch.randn(REQUESTS, 512))
        at.fill_(t)
        slots.copy_(table[:, 0].long() * PAGE + t)
        ids.copy_(torch.randint(-1, 3, (REQUESTS,)))
        target.copy_(torch.randint(0, 1000, (REQUESTS,)))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_gradient_through_autograd():
    z = torch.randn(7, 501, device="cuda", requires_grad=True)
    target = torch.randint(0, 501, (7,), device="cuda")
    lp, h = LogProbs.apply(z, target)
    w = torch.randn(2, 7, device="cuda")
    (w[0] * lp + w[1] * h).sum().backward()
    r = z.detach().double().requires_grad_()
    full = torch.log_softmax(r, 1)
    (w[0].double() * full.gather(1, target[:, None]).squeeze(1) - w[1].double() * (full.exp() * full).sum(1)).sum().backward()
    # p is off by (2 |ln p| + 6 + 2 |lse|) 2^-23 and the rest by 8 roundings of terms of at most |w| (1 + |ln p| + H)
    bound = 2.0 ** -23 * 60 * (w.abs().sum(0).double() * 20)[:, None] * torch.exp(full.detach()) + 2.0 ** -21 * w[0].abs().double()[:, None]
    assert ((z.grad.double() - r.grad).abs() <= bound + 1e-12).all()
    only = torch.randn(3, 50, device="cuda", requires_grad=True)
    LogProbs.apply(only, torch.zeros(3, device="cuda", dtype=torch.int64))[1].sum().backward()
    assert only.grad.isfinite().all()


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "many_requests.py")], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr
    assert "gradient norm" in r.stdout
