"""Log probabilities, entropy, alternatives and their gradient against float64.

Tolerances, u = 2^-23, m = max z, D = sum p |z - m|, S = sum e^(z - m).  An
exponential's argument is rounded twice and the hardware's 2^x by its unit: off
by a factor of 1 + (2 |z - m| + 4) u; a lane adds up to 64 terms a segment of
8192 values (fp32), and each join of two partial sums rounds four times, 16 of
them at most beyond one a segment.  So S is off by es = (2 D + 4 + 68 segments +
64) u of itself, ln S by es + 2 u |ln S|, log p_j = (z_j - m) - ln S by another
2 u (|z_j - m| + ln S), lse by 2 u (|m| + ln S), and the entropy, ln S - W / S, by
es (1 + 2 D) and 4 u (ln S + D).  A gradient's p is off by a factor of 1 + (2 |ln p| + 6 + 2 |lse|) u,
the rest by 8 roundings of terms of |g| + |e| (|ln p| + H); bf16 results by
2^-8 of themselves."""
import math

import pytest
import torch

import microscaling_block_quantization_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BF16, F32 = torch.bfloat16, torch.float32


def make(tokens, vocab, dtype, seed=0, masked=0.0, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * tokens + vocab)
    z = torch.randn(tokens, vocab, generator=g, device="cuda") * spread
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    if masked:
        z[torch.rand(tokens, vocab, generator=g, device="cuda") < masked] = -math.inf
    return z.to(dtype), target


def define(z):
    """m, lse, p and log p in float64, rows with something possible."""
    z = z.double()
    m = z.max(1, keepdim=True).values
    m = torch.where(m == -math.inf, 0.0, m)
    s = torch.exp(z - m).sum(1, keepdim=True)
    lp = (z - m) - torch.log(s)
    return m, torch.log(s), lp


def check(z, target, got, top=0, label=""):
    tokens, vocab = z.shape
    m, ln, lp = define(z)
    p = torch.exp(lp)
    d = torch.where(p > 0, (z.double() - m).abs(), 0.0)
    big_d = (p * d).sum(1)
    es = (2 * big_d + 4 + 68 * (-(-vocab // 8192) + 1) + 64) * U
    ln, m = ln.squeeze(1), m.squeeze(1)
    logprob, lse, entropy = (t.double() for t in got[:3])
    live = torch.isfinite(ln)
    assert (lse[~live] == -math.inf).all() and (entropy[~live] == 0).all(), f"{label}: rows of nothing"
    near = lambda a, b, tol, what: _near(a, b, tol, f"{label}: {what}")
    near(lse[live], (m + ln)[live], (es + 2 * U * (m.abs() + 2 * ln.abs()))[live], "lse")
    want = -torch.where(p > 0, p * lp, 0.0).sum(1)
    near(entropy[live], want[live], (es * (1 + 2 * big_d) + 4 * U * (ln.abs() + big_d))[live], "entropy")
    inside = (target >= 0) & (target < vocab)
    assert (logprob[~inside] == 0).all(), f"{label}: padding"
    at = target.clamp(0, vocab - 1)[:, None]
    of = lambda ids: (lp.gather(1, ids), (es + 2 * U * ln.abs())[:, None] + 2 * U * ((z.double().gather(1, ids) - m[:, None]).abs() + ln[:, None].abs()))
    w, tol = (t.squeeze(1) for t in of(at))
    use = inside & live
    near(logprob[use], w[use], tol[use], "logprob")
    assert (logprob[inside & ~live] == -math.inf).all()
    if not top:
        return
    values, ids = got[3:]
    order = torch.sort(z.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
    assert ids.dtype == torch.int64 and torch.equal(ids, order), f"{label}: alternatives"
    w, tol = of(order)
    assert (values[~live] == -math.inf).all()
    near(values.double()[live], w[live], tol[live], "top logprobs")


def _near(a, b, tol, label):
    same = a == b                                          # infinities
    err = torch.where(same, 0.0, (a - b).abs())
    tol = torch.where(same, 1.0, tol)
    assert (err <= tol).all(), f"{label}: {(err / tol).max().item():.2f} of the tolerance"


def run(tokens, vocab, dtype, top=0, label="", **kw):
    print(tokens, vocab, dtype, top, kw, flush=True)
    z, target = make(tokens, vocab, dtype, **kw)
    ws = mx.alloc_logprobs_workspace(tokens, vocab, top).fill_(0xFF)
    got = mx.mx_logprobs(z, target, top=top, workspace=ws)
    assert len(got) == (5 if top else 3)
    check(z, target, got, top, f"{tokens}x{vocab} top {top}")
    return z, target, got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 63, 64, 1000, 8191, 8192, 8193, 16385, 50001])
def test_vocabularies(vocab, dtype):
    """Rows that start at every alignment, end inside a piece, fill several segments."""
    for top in (0, 1, 5, 20, 64):
        if top <= vocab:
            run(11, vocab, dtype, top)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,vocab", [(1, 131072), (1, 300001), (2, 70000), (64, 40000), (700, 20000), (1023, 9000), (1024, 9000), (2500, 17001)])
def test_splits(tokens, vocab, dtype):
    run(tokens, vocab, dtype, 20)
    run(tokens, vocab, dtype, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [1, 7, 20, 64])
def test_masks(dtype, top):
    """Masked tokens, fewer possible ones than asked for, rows of nothing."""
    z, target = make(9, 33000, dtype, masked=0.5)
    z[1] = -math.inf
    z[2] = -math.inf
    z[2, 20000], z[2, 5] = 1.0, 1.0
    z[3] = -math.inf
    z[3, 32999] = -3.0
    z[4, 100:] = -math.inf
    z[5] = 0.25
    z[6, ::2], z[6, 1::2] = 0.0, -0.0
    check(z, target, mx.mx_logprobs(z, target, top=top), top)
    z, target = make(1500, 2000, dtype, masked=0.99)
    check(z, target, mx.mx_logprobs(z, target, top=top), top)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties_and_orders(dtype):
    """Many equal logits, rising and falling rows, all of the largest in one lane's places."""
    vocab = 40000
    z, target = make(8, vocab, dtype)
    z[0] = torch.randint(0, 3, (vocab,), device="cuda").to(dtype)
    z[1] = torch.linspace(-5, 5, vocab, device="cuda").to(dtype)
    z[2] = torch.linspace(5, -5, vocab, device="cuda").to(dtype)
    z[3] = (torch.arange(vocab, device="cuda") // 8 % 256 == 77).to(dtype) * 3 + z[3] * 1e-3
    z[4] = -z[4].abs()
    z[5, 39990:] = 9.0
    z[6, :70] = 9.0
    for top in (1, 20, 64):
        check(z, target, mx.mx_logprobs(z, target, top=top), top)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_logits(dtype):
    z, target = make(6, 5000, dtype)
    z[0] += 3e4
    z[1] *= 1e4
    z[2] = z[2] * 1e37
    z[3] *= 1e-30
    z[4, 17] = 3e38
    check(z, target, mx.mx_logprobs(z, target, top=9), 9)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [5, 1100])
def test_non_finite_rows_stay_alone(dtype, tokens):
    z, target = make(tokens, 20001, dtype)
    want = mx.mx_logprobs(z, target, top=20)
    z[1, 7], z[3, 20000] = math.nan, math.inf
    z[4] = math.nan
    target[4] = -100
    got = mx.mx_logprobs(z, target, top=20)
    keep = [0, 2] + list(range(5, tokens))
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    for i in (0, 1, 2, 3):
        assert got[i][[1, 3]].isnan().all()
    assert got[0][4] == 0 and got[1][4].isnan()
    assert (got[4] >= 0).all() and (got[4] <= 20000).all()


def test_padding_views_and_same_bits():
    z, target = make(40, 5003, BF16)
    target[::3] = torch.tensor([-100, -1, 5003, 2 ** 40], device="cuda").repeat(4)[:14]
    want = mx.mx_logprobs(z, target, top=20)
    check(z, target, want, 20)
    wide = torch.full((41, 5100), float("nan"), device="cuda", dtype=BF16)
    wide[:40, 8:5011] = z
    view = mx.mx_logprobs(wide[:40, 8:5011], target, top=20)
    check(z, target, view, 20)                             # rows elsewhere against 16 bytes: sums in another order
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(mx.mx_logprobs(wide[:40, 8:5011], target, top=20), view))
        assert all(torch.equal(a, b) for a, b in zip(mx.mx_logprobs(z, target, top=20), want))
    empty = mx.mx_logprobs(z[:0], target[:0], top=3)
    assert empty[0].shape == (0,) and empty[4].shape == (0, 3)


def test_rows_past_32_bits():
    z = torch.zeros(40000, 60000, device="cuda", dtype=BF16)
    assert z.numel() * 2 > 1 << 32
    z[-2:] = torch.randn(2, 60000, device="cuda").to(BF16)
    target = torch.full((40000,), 123, device="cuda")
    got = mx.mx_logprobs(z, target, top=5)
    check(z[-2:], target[-2:], [t[-2:] for t in got], 5)
    dz = mx.mx_logprobs_backward(torch.ones(40000, device="cuda"), None, z, target, got[1])
    grad_check(z[-2:], target[-2:], torch.ones(2, device="cuda"), None, got[1][-2:], None, dz[-2:])


# ---- the gradient -----------------------------------------------------------------
def grad_check(z, target, gl, gh, lse, entropy, dz, label=""):
    z64 = z.double()
    lp = z64 - lse.double()[:, None]
    p = torch.exp(lp)
    g = (torch.zeros(z.shape[0], device="cuda") if gl is None else gl).double()[:, None]
    e = (torch.zeros(z.shape[0], device="cuda") if gh is None else gh).double()[:, None]
    h = (torch.zeros(z.shape[0], device="cuda") if entropy is None else entropy).double()[:, None]
    inside = (target >= 0) & (target < z.shape[1])
    g = g * inside[:, None]
    lp0 = torch.where(p > 0, lp, 0.0)
    want = -p * (g + e * (lp0 + h))
    one = torch.zeros_like(want).scatter_(1, target.clamp(0, z.shape[1] - 1)[:, None], 1.0)
    want = want + g * one
    dead = lse == -math.inf
    want[dead] = 0
    tol = U * ((2 * lp0.abs() + 6 + 2 * lse.double()[:, None].abs()) + 8) * p * (g.abs() + e.abs() * (lp0.abs() + h.abs())) + 2 * U * g.abs() * one
    tol[dead] = 0
    # the hardware's exponential gives 0 below 2^-126
    tol = tol + 2.0 ** -125 * (g.abs() + e.abs() * (200 + h.abs()))
    if dz.dtype == BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    err = (dz.double() - want).abs()
    assert dz.dtype == z.dtype and (err <= tol).all(), f"{label}: {(err / tol).max().item():.2f} of the tolerance"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [1, 5, 8, 1003, 8192, 20001])
def test_gradient(vocab, dtype):
    z, target = make(13, vocab, dtype, masked=0.2 if vocab > 100 else 0.0)
    target[3], target[4] = -100, vocab
    if vocab > 100:
        z[5] = -math.inf
    _, lse, entropy = mx.mx_logprobs(z, target)
    gl, gh = torch.randn(13, device="cuda"), torch.randn(13, device="cuda")
    for a, b in ((gl, gh), (gl, None), (None, gh), (None, None)):
        dz = mx.mx_logprobs_backward(a, b, z, target, lse, entropy)
        grad_check(z, target, a, b, lse, entropy, dz, f"{vocab}")
    dz = mx.mx_logprobs_backward(gl, gh, z, target, lse, entropy)
    own = z.clone()
    assert mx.mx_logprobs_backward(gl, gh, own, target, lse, entropy, d_logits=own) is own and torch.equal(own, dz)
    wide = torch.full((14, vocab + 9), 7.0, device="cuda", dtype=dtype)
    out = wide[:13, 8:8 + vocab]
    mx.mx_logprobs_backward(gl, gh, z, target, lse, entropy, d_logits=out)
    assert torch.equal(out, dz) and (wide[13] == 7).all() and (wide[:, :8] == 7).all() and (wide[:, 8 + vocab:] == 7).all()


def test_gradient_against_differences():
    """Both outputs' sum, differenced in float64 from the definition and in fp32 through the forward call."""
    z, target = make(4, 37, F32)
    gl, gh = torch.randn(4, device="cuda"), torch.randn(4, device="cuda")

    def value(x):
        m, ln, lp = define(x)
        p = torch.exp(lp)
        return (gl.double() * lp.gather(1, target[:, None]).squeeze(1) - gh.double() * (p * lp).sum(1)).sum()

    _, lse, entropy = mx.mx_logprobs(z, target)
    dz = mx.mx_logprobs_backward(gl, gh, z, target, lse, entropy).double()
    h = 1e-5
    for j in range(37):
        for t in range(4):
            up, down = z.double(), z.double()
            up[t, j] += h
            down[t, j] -= h
            # the difference's own error: h^2 of third derivatives below 30, and 1e-16 / h
            assert abs((value(up) - value(down)) / (2 * h) - dz[t, j]) < 1e-5 * (1 + gl.abs().max() + gh.abs().max())
    step = 1e-2                                            # h^2 / 6 of a third derivative below 30, sums of 6 in fp32 over 2 h
    for j in (0, 11, 36):
        up, down = z.clone(), z.clone()
        up[:, j] += step
        down[:, j] -= step
        a, b = mx.mx_logprobs(up, target), mx.mx_logprobs(down, target)
        num = (gl * (a[0] - b[0]) + gh * (a[2] - b[2])) / (2 * step)
        assert ((num - dz[:, j].float()).abs() < 2e-3 * (1 + gl.abs() + gh.abs())).all()


def test_graph_streams_and_a_shared_workspace():
    z, target = make(6, 60000, BF16)
    ws = mx.alloc_logprobs_workspace(1024, 70000, 30)
    mx.mx_logprobs(z, target, top=20, workspace=ws)
    g = torch.cuda.CUDAGraph()
    gl = torch.randn(6, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = mx.mx_logprobs(z, target, top=20, workspace=ws)
        dz = mx.mx_logprobs_backward(gl, got[2], z, target, got[1], got[2])
    for i in range(4):
        z.copy_(torch.randn(6, 60000))
        target.copy_(torch.randint(0, 60000, (6,)))
        g.replay()
        torch.cuda.synchronize()
        want = mx.mx_logprobs(z, target, top=20)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(dz, mx.mx_logprobs_backward(gl, want[2], z, target, want[1], want[2]))
        check(z, target, got, 20)
    torch.cuda.synchronize()
    outs = [mx.mx_logprobs(z, target, top=20, stream=s) for s in [torch.cuda.Stream() for _ in range(4)]]
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, got))
    with pytest.raises(mx.MxError):
        mx.mx_logprobs(z, target, top=20, workspace=mx.alloc_logprobs_workspace(6, 60000, 19).clone()[:64])
