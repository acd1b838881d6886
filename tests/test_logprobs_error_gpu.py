"""How far log probabilities, lse and entropy lie from float64 on average: a bound
on the root mean square over many rows, which a loss of a few bits anywhere
passes, where the worst case's bound of every rounding at once would not see it.

u = 2^-23, roundings independent and of mean 0, each of rms 0.29 u at most of its
result.  With m = max z, S = sum e^(z - m), W = sum e^(z - m) (z - m) and
D = -W / S: a lane adds 16 (fp32) or 32 (bf16) terms, its segments, the 64 lanes,
4 waves and up to 64 lanes of splits join in at most 24 steps of 4 roundings, so S
is off by sqrt(32 + 96) 0.29 u = 3.3 u of itself, W likewise with one more
product a term, together less than 5 u; the exponentials' errors are averaged
over the terms, and at most (D + 2) u where one term or one value is all there is.
ln S rounds by a unit of the logarithm and a product with ln 2, u of it, and each
result by its own sum of two terms, half a unit of the larger:
  lse:      5 u + (D + 2) u + u ln S + u (|m| + ln S)
  log p:    5 u + (D + 2) u + u ln S + u (|z - m| + ln S)
  entropy:  (5 + D + 2) u (1 + D) + u ln S + u (ln S + D)."""
import pytest
import torch

import microscaling_block_quantization_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,vocab", [(512, 50001), (256, 131072), (1500, 20000)])
@pytest.mark.parametrize("spread,offset", [(0.5, 0.0), (2.5, 0.0), (2.5, -100.0), (6.0, 300.0)])
def test_rms(dtype, tokens, vocab, spread, offset):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = (torch.randn(tokens, vocab, generator=g, device="cuda") * spread + offset).to(dtype)
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    logprob, lse, entropy = mx.mx_logprobs(z, target)
    z = z.double()
    m = z.max(1).values
    e = torch.exp(z - m[:, None])
    s = e.sum(1)
    d = -(e * (z - m[:, None])).sum(1) / s
    zt, ln = z.gather(1, target[:, None]).squeeze(1) - m, torch.log(s)
    rms = lambda t: t.pow(2).mean().sqrt().item()
    common = (5 + d + 2) * U + U * ln
    for name, got, want, room in (("lse", lse, m + ln, common + U * (m.abs() + ln)),
                                  ("log p", logprob, zt - ln, common + U * (zt.abs() + ln)),
                                  ("entropy", entropy, ln + d, (5 + d + 2) * U * (1 + d) + U * ln + U * (ln + d))):
        off, most = rms(got.double() - want), rms(room)
        print(f"{name} {off / most:.3f}", end=" ")
        assert off <= most, f"{name}: {off / most:.2f} of the tolerance"
