"""Low-rank adapters of many requests against float64.

Tolerance, u = 2^-23.  h = a x sums K products in fp32 (bf16 products are
exact, fp32 ones off by u): off by at most (K + 24) u |a| |x|.  scale and the
second product's sum over rank values in three parts: (3 rank + 24) u of
s |b| |h|.  Adding the base: u of the result.  A bf16 output adds 2^-8 of its
magnitude."""
import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BF16, F32 = torch.bfloat16, torch.float32


def make(tokens, n, k, rank, count, dtype=BF16, base=BF16, seed=0, scales=True):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens + n)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    a, b = (r(count, rank, k) * k ** -0.5).to(dtype), (r(count, n, rank) * 0.3).to(dtype)
    ad = mx.Adapters(a, b, torch.rand(count, generator=g, device="cuda") + 0.5 if scales else None)
    ids = torch.randint(-1, count, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    return ad, r(tokens, k).to(dtype), ids, None if base is None else r(tokens, n).to(base)


def check(ad, x, ids, base, y, label=""):
    count, rank, k = ad.a.shape
    x64, n = x.double(), ad.b.shape[1]
    want = torch.zeros(x.shape[0], n, device="cuda", dtype=torch.float64) if base is None else base.double().clone()
    tol = torch.zeros_like(want)
    for i in range(count):
        at = torch.nonzero(ids == i).squeeze(1)
        if not len(at):
            continue
        a, b = ad.a[i].double(), ad.b[i].double()
        s = 1.0 if ad.scales is None else float(ad.scales[i])
        h, size = torch.mm(x64[at], a.t().contiguous()), torch.mm(x64[at].abs(), a.abs().t().contiguous())
        want[at] += s * torch.mm(h, b.t().contiguous())
        tol[at] += s * torch.mm((k + 24) * U * size + (3 * rank + 24) * U * h.abs(), b.abs().t().contiguous())
    tol += 2 * U * want.abs()
    if y.dtype == BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    err = (y.double() - want).abs()
    assert (err <= tol).all(), f"{label}: {(err / tol.clamp(min=1e-300)).max().item():.2f} of the tolerance"


def run(tokens, n, k, rank, count, dtype=BF16, base=BF16, out=None, **kw):
    print(tokens, n, k, rank, count, dtype, base, out, flush=True)
    ad, x, ids, b = make(tokens, n, k, rank, count, dtype, base, **kw)
    ws = mx.alloc_lora_workspace(ad, tokens).fill_(0xFF)
    y = mx.mx_lora(x, ad, ids, b, out_dtype=out, workspace=ws)
    assert y.dtype == (out or base or dtype)
    check(ad, x, ids, b, y, f"{tokens}x{n}x{k} rank {rank}")
    return ad, x, ids, b, y


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranks(rank, dtype):
    run(1, 200, 256, rank, 3, dtype)
    run(7, 129, 1032, rank, 5, dtype, F32, F32)
    run(50, 320, 264, rank, 4, dtype)


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 31, 33, 64, 65, 200, 1025])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tokens(tokens, dtype):
    run(tokens, 256, 512, 16, 6, dtype)
    run(tokens, 100, 2048, 8, 40, dtype, None, F32)


@pytest.mark.parametrize("n", [1, 3, 15, 16, 17, 63, 64, 65, 255, 1000, 4097])
def test_outputs(n):
    """Rows that end inside a tile, rows that start at no multiple of 16 bytes."""
    for base in (BF16, F32, None):
        for out in (BF16, F32):
            run(5, n, 128, 16, 3, BF16, base, out)
            run(40, n, 128, 32, 3, BF16, base, out)


@pytest.mark.parametrize("k", [8, 24, 120, 128, 136, 1024, 4096, 8200])
def test_inputs(k):
    run(3, 64, k, 16, 2)
    run(70, 64, k, 16, 2)
    run(3, 64, k, 16, 2, F32)


def test_no_scales_and_one_adapter():
    run(20, 64, 256, 16, 1, scales=False)
    run(1, 64, 256, 16, 1, scales=False)
    run(100, 64, 256, 64, 1, F32)


def test_prompts_side_by_side():
    ad, x, ids, base = make(500, 300, 512, 16, 5)
    ids = torch.repeat_interleave(torch.tensor([3, -1, 0, 4, 4], device="cuda", dtype=torch.int32),
                                  torch.tensor([33, 100, 200, 1, 166], device="cuda"))
    check(ad, x, ids, base, mx.mx_lora(x, ad, ids, base))


@pytest.mark.parametrize("tokens", [5, 300])
def test_tokens_without_an_adapter(tokens):
    """Any id outside the adapters leaves the base, whatever the token holds."""
    ad, x, ids, base = make(tokens, 200, 256, 16, 4)
    ids[0], ids[1], ids[2] = -1, 4, 2 ** 31 - 1
    ids[3] = -2 ** 31
    x[:4] = float("nan")
    y = mx.mx_lora(x, ad, ids, base)
    assert torch.equal(y[:4], base[:4])
    check(ad, x[4:], ids[4:], base[4:], y[4:])
    none = mx.Adapters(ad.a[:0], ad.b[:0], ad.scales[:0])
    assert torch.equal(mx.mx_lora(x, none, ids, base), base)
    assert (mx.mx_lora(x, none, ids, None) == 0).all()


def test_non_finite_tokens_stay_alone():
    ad, x, ids, base = make(18, 100, 256, 16, 3)
    ids.copy_(torch.arange(18) % 3)
    want = mx.mx_lora(x, ad, ids, base)
    x[4, 7], x[9, 0] = float("nan"), float("inf")
    y = mx.mx_lora(x, ad, ids, base)
    keep = [t for t in range(18) if t not in (4, 9)]
    assert torch.equal(y[keep], want[keep]) and y[4].isnan().all() and not y[9].isfinite().any()


@pytest.mark.parametrize("tokens", [12, 40])
@pytest.mark.parametrize("rank,dtype", [(8, BF16), (16, BF16), (72, BF16), (16, F32)])
def test_non_finite_adapters_stay_alone(tokens, rank, dtype):
    """NaN and Inf in an adapter's weights or scale reach the tokens that name it, not others beside them."""
    ad, x, ids, base = make(tokens, 100, 256, rank, 4, dtype, dtype)
    ids.copy_(torch.arange(tokens) % 5 - 1)
    want = mx.mx_lora(x, ad, ids, base)
    ad.a[1, 3, 7], ad.b[2, :, 1] = float("nan"), float("inf")
    ad.scales[3] = float("nan")
    y = mx.mx_lora(x, ad, ids, base)
    clean = (ids <= 0).nonzero().squeeze(1)
    assert torch.equal(y[clean], want[clean])
    assert y[ids == 1].isnan().all() and not y[ids == 2].isfinite().any() and y[ids == 3].isnan().all()


def test_huge_and_tiny_values():
    """Rank values far from one keep their bits in the three parts."""
    ad, x, ids, base = make(9, 64, 128, 16, 2, BF16, None)
    for e in (-50, 40):
        y = mx.mx_lora((x.float() * 2.0 ** e).to(BF16), ad, ids, None, out_dtype=F32)
        check(ad, (x.float() * 2.0 ** e).to(BF16), ids, None, y, f"2^{e}")


def test_views_in_place_and_same_bits():
    ad, x, ids, base = make(37, 136, 256, 16, 4)
    want = mx.mx_lora(x, ad, ids, base)
    wide = torch.full((37, 3, 256), 9.0, device="cuda", dtype=BF16)
    wide[:, 1] = x
    out = torch.full((40, 200), 5.0, device="cuda", dtype=BF16)
    for _ in range(3):
        assert mx.mx_lora(wide[:, 1], ad, ids, base, y=out[:37, 8:144]) is not None
        assert torch.equal(out[:37, 8:144], want)
    assert (out[37:] == 5).all() and (out[:, :8] == 5).all() and (out[:, 144:] == 5).all()
    again = base.clone()
    assert mx.mx_lora(x, ad, ids, again, y=again) is again and torch.equal(again, want)
    assert mx.mx_lora(x[:0], ad, ids[:0], base[:0]).shape == (0, 136)


def test_beside_the_shared_projection():
    """A decode batch and a prompt: the 4-bit product, then the adapters on it."""
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(320, 512, generator=g, device="cuda").to(BF16)
    qw, dw, _ = mx.mx_quantize(mx.MXFP4, w, dequant=F32)
    for tokens in (3, 128):
        ad, x, ids, _ = make(tokens, 320, 512, 16, 4, base=None)
        if tokens <= 16:
            base = mx.mx_matvec(mx.MXFP4, qw, x, out_dtype=F32)
        else:
            qx, _, _ = mx.mx_quantize(mx.MXFP8_E4M3, x)
            base = mx.mx_gemm(mx.MXFP8_E4M3, qx, mx.MXFP4, qw, out_dtype=F32)
        check(ad, x, ids, base, mx.mx_lora(x, ad, ids, base, out_dtype=BF16))


def test_workspace_of_a_larger_call():
    ad, x, ids, base = make(200, 64, 4096, 16, 4)
    big = mx.alloc_lora_workspace(ad, 200).fill_(0xFF)
    for t in (1, 16, 17, 63, 64, 65, 100, 200):
        assert mx.mx_lora_workspace_size(ad, t) <= big.numel()
        got = mx.mx_lora(x[:t], ad, ids[:t], base[:t], workspace=big)
        check(ad, x[:t], ids[:t], base[:t], got)
    with pytest.raises(mx.MxError):
        mx.mx_lora(x, ad, ids, base, workspace=big[:-256].clone())


def test_graph_and_streams():
    """A captured call follows its ids, tokens and base; calls on several streams at once."""
    ad, x, ids, base = make(12, 256, 512, 16, 6)
    ws = mx.alloc_lora_workspace(ad, 12)
    mx.mx_lora(x, ad, ids, base, workspace=ws)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = mx.mx_lora(x, ad, ids, base, workspace=ws)
    for i in range(4):
        ids.copy_(torch.randint(-1, 6, (12,)))
        x.copy_(torch.randn_like(x))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mx.mx_lora(x, ad, ids, base))
    want = mx.mx_lora(x, ad, ids, base)
    torch.cuda.synchronize()
    got = [mx.mx_lora(x, ad, ids, base, stream=s) for s in [torch.cuda.Stream() for _ in range(4)]]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


def test_offsets_past_32_bits():
    """Adapters of over 4 GiB, the last one in use; a base of over 2^32 bytes."""
    count, rank, k, n = 300, 256, 32768, 64
    a = torch.empty(count, rank, k, device="cuda", dtype=BF16)
    assert a.numel() * 2 > 1 << 32
    b = torch.empty(count, n, rank, device="cuda", dtype=BF16)
    a[-1], b[-1] = torch.randn(rank, k, device="cuda") * 0.01, torch.randn(n, rank, device="cuda")
    x = torch.randn(2, k, device="cuda").to(BF16)
    ids = torch.tensor([-1, count - 1], device="cuda", dtype=torch.int32)
    y = mx.mx_lora(x, mx.Adapters(a, b), ids, None, out_dtype=F32)
    check(mx.Adapters(a[-1:].clone(), b[-1:].clone()), x, torch.tensor([-1, 0], device="cuda"), None, y)
    del a
    ad, x, ids, _ = make(70000, 64, 128, 8, 3)
    wide = torch.zeros(70000, 40000, device="cuda", dtype=BF16)
    assert wide.numel() * 2 > 1 << 32
    y = mx.mx_lora(x, ad, ids, wide[:, 8:72], y=wide[:, 8:72])
    check(ad, x[-500:], ids[-500:], torch.zeros(500, 64, device="cuda", dtype=BF16), y[-500:])
