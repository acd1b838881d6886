"""Norm and rotation of query and key heads (mx_qk_rope) and its gradient
against the formulas in float64.

Tolerances, u = 2^-23.  A value u_a = w x rstd carries at most (D/2 + 16) u/2
of relative error (the sum of D squares, the square root, three products), so
an output is off by at most (D/2 + 32) u (|u_a| + |u_b|).  An input gradient
rstd (h - n mean(h n)) is off by at most (D + 64) u rstd (|h_a| + |h_b| +
|n| mean|h n|) with |h| taken over the pair.  A weight gradient is a sum over
R head vectors: (R + D + 64) u sum |g n|, |g| over the pair.  A bf16 output
adds 2^-8 of its magnitude."""
import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


def pair_index(dim, rot, adjacent):
    """partner[i] and sign: y_i = u_i cos + sign u_partner sin (0 unrotated); angle column of i"""
    partner, sign, col = np.arange(dim), np.zeros(dim), np.zeros(dim, int)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
        partner[a], partner[b], sign[a], sign[b], col[a], col[b] = b, a, -1, 1, i, i
    return partner, sign, col


class Case:
    def __init__(self, t, hq, hk, dim, rot, dtype, adjacent=False, weights=True, w_dtype=None, rows=97, seed=0, fused=True):
        g = torch.Generator(device="cuda").manual_seed(seed + 1000 * dim + t)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.t, self.hq, self.hk, self.dim, self.rot, self.adjacent = t, hq, hk, dim, rot, adjacent
        both = r(t, hq + hk + 1, dim).to(dtype)             # one more head in between, as values would lie
        self.q, self.k = both[:, :hq], both[:, hq + 1:]
        if not fused:
            self.q, self.k = self.q.contiguous(), self.k.contiguous()
        ang = torch.rand(rows, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 6.3
        self.cos, self.sin = ang.cos().float(), ang.sin().float()
        self.pos = torch.randint(0, rows, (t,), generator=g, device="cuda", dtype=torch.int32)
        wd = w_dtype or dtype
        self.qw = (1 + 0.3 * r(dim)).to(wd) if weights else None
        self.kw = (1 + 0.3 * r(dim)).to(wd) if weights else None
        self.dq, self.dk = r(t, hq, dim).to(dtype), r(t, hk, dim).to(dtype)
        self.eps = 1e-5

    def args(self):
        return dict(cos=self.cos, sin=self.sin, positions=self.pos, q_weight=self.qw, k_weight=self.kw, eps=self.eps,
                    interleaved=self.adjacent)

    def tables(self):
        partner, sign, col = pair_index(self.dim, self.rot, self.adjacent)
        p = self.pos.cpu().numpy()
        turned = (sign != 0)[None, None]
        if self.rot == 0:
            return partner, np.ones((self.t, 1, self.dim)), np.zeros((self.t, 1, self.dim))
        c = np.where(turned, self.cos.double().cpu().numpy()[p][:, None, col], 1.0)
        s = np.where(turned, self.sin.double().cpu().numpy()[p][:, None, col] * sign, 0.0)
        return partner, c, s

    def forward64(self, x, w):
        partner, c, s = self.tables()
        x = x.double().cpu().numpy() if isinstance(x, torch.Tensor) else x
        if w is not None:
            rstd = (np.mean(x * x, -1, keepdims=True) + self.eps) ** -0.5
            u = x * rstd * w.double().cpu().numpy()
        else:
            u = x
        return u * c + u[..., partner] * s, np.abs(u) + np.abs(u[..., partner])

    def backward64(self, dy, x, w):
        partner, c, s = self.tables()
        dy, x = dy.double().cpu().numpy(), x.double().cpu().numpy()
        back = (dy * s)[..., partner]                      # the transpose of the turn
        g = dy * c + back
        ga = np.abs(dy) + np.abs(dy[..., partner])
        if w is None:
            return g, ga, None, None
        w = w.double().cpu().numpy()
        rstd = (np.mean(x * x, -1, keepdims=True) + self.eps) ** -0.5
        n, h, ha = x * rstd, g * w, ga * np.abs(w)
        dx = rstd * (h - n * np.mean(h * n, -1, keepdims=True))
        mag = rstd * (ha + np.abs(n) * np.mean(ha * np.abs(n), -1, keepdims=True))
        return dx, mag, (g * n).sum((0, 1)), (ga * np.abs(n)).sum((0, 1))


def near(got, want, tol, label):
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{label}: {np.max(err / np.maximum(tol, 1e-300)):.2f} of the tolerance"


SHAPES = [(1, 32, 8, 128, 128), (3, 4, 4, 64, 64), (17, 5, 1, 96, 64), (2, 3, 2, 256, 256), (5, 2, 1, 512, 128), (2, 1, 1, 1024, 1024),
          (9, 3, 1, 80, 20), (4, 2, 2, 8, 8), (3, 2, 1, 24, 0), (6, 7, 3, 128, 0), (5, 4, 2, 72, 70), (33, 6, 2, 192, 96),
          (2, 3, 3, 1000, 998), (11, 9, 5, 16, 16)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("adjacent", [False, True])
def test_forward_and_backward(shape, dtype, adjacent):
    print(shape, dtype, adjacent, flush=True)
    for weights in (True, False):
        c = Case(*shape, dtype, adjacent, weights)
        yq, yk = mx.mx_qk_rope(c.q, c.k, **c.args())
        for y, x, w, what in ((yq, c.q, c.qw, "q"), (yk, c.k, c.kw, "k")):
            want, mag = c.forward64(x, w)
            near(y, want, (c.dim / 2 + 32) * U * mag, what)
        dq, dk, dqw, dkw = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
        for d, dw, dy, x, w, what in ((dq, dqw, c.dq, c.q, c.qw, "dq"), (dk, dkw, c.dk, c.k, c.kw, "dk")):
            want, mag, w64, wmag = c.backward64(dy, x, w)
            near(d, want, (c.dim + 64) * U * mag, what)
            if w is None:
                assert dw is None
            else:
                assert dw.dtype == torch.float32
                near(dw, w64, (c.t * x.shape[1] + c.dim + 64) * U * wmag, what + " weight")


@pytest.mark.parametrize("t", [257, 2100])
@pytest.mark.parametrize("w_dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_and_weight_types(t, w_dtype):
    """More head vectors than workgroups hold at once, weights of either type."""
    c = Case(t, 12, 4, 64, 64, torch.bfloat16, w_dtype=w_dtype, fused=False)
    yq, yk = mx.mx_qk_rope(c.q, c.k, **c.args())
    near(yq, c.forward64(c.q, c.qw)[0], (c.dim / 2 + 32) * U * c.forward64(c.q, c.qw)[1], "q")
    got = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    for d, dw, dy, x, w in ((got[0], got[2], c.dq, c.q, c.qw), (got[1], got[3], c.dk, c.k, c.kw)):
        want, mag, w64, wmag = c.backward64(dy, x, w)
        near(d, want, (c.dim + 64) * U * mag, "dx")
        near(dw, w64, (c.t * x.shape[1] + c.dim + 64) * U * wmag, "dw")
    again = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "the same inputs gave other bits"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_than_the_cache_holds(dtype):
    """A launch that writes past L2 (over 32 MiB) and takes several heads per
    lane gives what slices of its tokens give, bit for bit; the weight sums to
    the rounding of their order."""
    t, hq, hk, dim = 4700, 30, 7, 128
    assert t * (hq + hk) * dim * 2 > 32 << 20
    c = Case(t, hq, hk, dim, dim, dtype)
    yq, yk = mx.mx_qk_rope(c.q, c.k, **c.args())
    dq, dk, dqw, dkw = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    sums = [torch.zeros(dim, device="cuda", dtype=torch.float64) for _ in range(2)]
    for a in range(0, t, 470):
        part = slice(a, a + 470)
        args = c.args() | dict(positions=c.pos[part].contiguous())
        sq, sk = mx.mx_qk_rope(c.q[part], c.k[part], **args)
        assert torch.equal(sq, yq[part]) and torch.equal(sk, yk[part])
        gq, gk, gqw, gkw = mx.mx_qk_rope_backward(c.dq[part], c.dk[part], c.q[part], c.k[part], **args)
        assert torch.equal(gq, dq[part]) and torch.equal(gk, dk[part])
        sums[0] += gqw.double()
        sums[1] += gkw.double()
    for dw, total, dy, x, w in ((dqw, sums[0], c.dq, c.q, c.qw), (dkw, sums[1], c.dk, c.k, c.kw)):
        wmag = c.backward64(dy, x, w)[3]
        near(dw, total.cpu().numpy(), 2 * (t * x.shape[1] + dim + 64) * U * wmag, "dw")


@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 40)])
def test_in_place_queries_only_and_mixed_weights(dim, rot):
    c = Case(21, 6, 2, dim, rot, torch.bfloat16)
    yq, yk = mx.mx_qk_rope(c.q, c.k, **c.args())
    q, k = c.q.clone(), c.k.clone()
    mx.mx_qk_rope(q, k, q_out=q, k_out=k, **c.args())
    assert torch.equal(q, yq) and torch.equal(k, yk)
    a = c.args()
    a["k_weight"] = None
    only, none = mx.mx_qk_rope(c.q, None, **a)
    assert none is None and torch.equal(only, yq)
    _, plain = mx.mx_qk_rope(c.q, c.k, **a)                 # queries normed, keys only turned
    want, mag = c.forward64(c.k, None)
    near(plain, want, (dim / 2 + 32) * U * mag, "k without norm")
    dq, dk, dqw, dkw = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    gq, gk = c.dq.clone(), c.dk.clone()
    mx.mx_qk_rope_backward(gq, gk, c.q, c.k, dq=gq, dk=gk, **c.args())
    assert torch.equal(gq, dq) and torch.equal(gk, dk)
    oq, ok, oqw, okw = mx.mx_qk_rope_backward(c.dq, None, c.q, None, **a)
    assert ok is None and okw is None and torch.equal(oq, dq) and torch.equal(oqw, dqw)


@pytest.mark.parametrize("dim", [64, 72])
def test_positions_outside_the_table_and_no_tokens(dim):
    c = Case(6, 3, 2, dim, 32, torch.float32)
    c.pos[1], c.pos[4] = -1, 97
    yq, yk = mx.mx_qk_rope(c.q, c.k, **c.args())
    for y in (yq, yk):
        assert y[[1, 4], :, :32].isnan().all() and y[[0, 2, 3, 5]].isfinite().all()
        assert y[:, :, 32:].isfinite().all()
    dq, dk, _, _ = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    assert dq[[1, 4]].isnan().all() and dq[[0, 2, 3, 5]].isfinite().all() and dk[[0, 2, 3, 5]].isfinite().all()
    e = Case(0, 3, 2, dim, 32, torch.float32)
    yq, yk = mx.mx_qk_rope(e.q, e.k, **e.args())
    assert yq.shape == (0, 3, dim)
    _, _, dqw, dkw = mx.mx_qk_rope_backward(e.dq, e.dk, e.q, e.k, **e.args())
    assert (dqw == 0).all() and (dkw == 0).all()


def test_zero_and_non_finite_heads():
    c = Case(4, 2, 2, 128, 128, torch.float32, fused=False)
    c.q[0, 0] = 0
    c.q[1, 1, 5] = float("nan")
    c.k[2, 0, 7] = float("inf")
    yq, yk = mx.mx_qk_rope(c.q, c.k, **c.args())
    assert (yq[0, 0] == 0).all() and yq[1, 1].isnan().all() and yk[2, 0].isnan().any()
    yq[1, 1], yk[2, 0] = 0, 0
    assert yq.isfinite().all() and yk.isfinite().all()
    c.q[1, 1], c.k[2, 0] = 1, 1
    got = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    want, mag, _, _ = c.backward64(c.dq, c.q, c.qw)
    near(got[0], want, (c.dim + 64) * U * mag, "dq with a zero head")


@pytest.mark.parametrize("dim,rot,adjacent", [(64, 64, False), (96, 32, True), (40, 20, False)])
def test_gradient_against_differences(dim, rot, adjacent):
    """Along one direction v: (L(x + hv) - L(x - hv)) / 2h of the kernel's own
    forward, L = sum dy y.  It is off by the difference's own truncation (taken
    in float64) and by the rounding of the two outputs over 2h."""
    c = Case(7, 3, 2, dim, rot, torch.float32, adjacent, fused=False)
    g = torch.Generator(device="cuda").manual_seed(3)
    vq, vk = (torch.randn(x.shape, generator=g, device="cuda") for x in (c.q, c.k))
    vw = torch.randn(dim, generator=g, device="cuda")
    h = 2.0 ** -7
    dq, dk, dqw, dkw = mx.mx_qk_rope_backward(c.dq, c.dk, c.q, c.k, **c.args())
    slope = sum((a.double() * b.double()).sum().item() for a, b in ((dq, vq), (dk, vk), (dqw, vw), (dkw, vw)))

    def loss(sign):
        q, k = c.q + sign * h * vq, c.k + sign * h * vk
        a = c.args() | dict(q_weight=c.qw + sign * h * vw, k_weight=c.kw + sign * h * vw)
        yq, yk = mx.mx_qk_rope(q, k, **a)
        own = (yq.double() * c.dq.double()).sum().item() + (yk.double() * c.dk.double()).sum().item()
        exact, mag = 0.0, 0.0
        for x, w, dy in ((q, a["q_weight"], c.dq), (k, a["k_weight"], c.dk)):
            y, m = c.forward64(x, w)
            dy = dy.double().cpu().numpy()
            exact += (dy * y).sum()
            mag += (np.abs(dy) * m).sum()
        return own, exact, mag

    (op, ep, mp), (om, em, mm) = loss(1), loss(-1)
    s64 = 0.0
    for dy, x, w, v in ((c.dq, c.q, c.qw, vq), (c.dk, c.k, c.kw, vk)):
        dx, _, dw, _ = c.backward64(dy, x, w)
        s64 += (dx * v.double().cpu().numpy()).sum() + (dw * vw.double().cpu().numpy()).sum()
    truncation = abs((ep - em) / (2 * h) - s64)
    rounding = (dim / 2 + 32) * U * (mp + mm) / (2 * h)
    # x + hv and w + hv are rounded too: at most u/2 of each, through the slope's own magnitudes
    moved = U * (mp + mm) / (2 * h)
    assert truncation < 0.05 * abs(s64) + 1.0
    assert abs((op - om) / (2 * h) - slope) <= truncation + rounding + moved + (dim + 64) * U * (mp + mm)
