"""examples/decode_step.py's Function around mx_qk_rope and its gradient: every
choice of key and weights against torch's own autograd in float64.  fp32
throughout, so a few hundred roundings of 2^-24 on sums of like size."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain(x, w, c, s):
    u = x if w is None else x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    a, b = u[..., :32], u[..., 32:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


@pytest.mark.parametrize("key,k_weight", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("q_weight", [True, False])
def test_key_and_weights_may_be_missing(key, k_weight, q_weight):
    from decode_step import QKRope, rotation_tables
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k = r(9, 4, 64), r(9, 2, 64) if key else None
    qw, kw = 1 + 0.1 * r(64) if q_weight else None, 1 + 0.1 * r(64) if k_weight else None
    leaves = [q, k, qw, kw]
    mine = [None if t is None else t.clone().requires_grad_() for t in leaves]
    ref = [None if t is None else t.double().cpu().requires_grad_() for t in leaves]
    cos, sin = rotation_tables(32, 64, torch.device("cuda"))
    pos = torch.arange(9, device="cuda", dtype=torch.int32) * 3
    tq, tk = r(9, 4, 64), r(9, 2, 64)
    yq, yk = QKRope.apply(mine[0], mine[1], cos, sin, pos, mine[2], mine[3], 1e-6)
    loss = ((yq - tq) ** 2).sum() + (((yk - tk) ** 2).sum() if key else 0)
    loss.backward()
    c, s = (t.double().cpu()[pos.cpu().long()][:, None] for t in (cos, sin))
    want = ((plain(ref[0], ref[2], c, s) - tq.double().cpu()) ** 2).sum()
    if key:
        want = want + ((plain(ref[1], ref[3], c, s) - tk.double().cpu()) ** 2).sum()
    want.backward()
    for m, e in zip(mine, ref):
        if m is not None:
            assert (m.grad.double().cpu() - e.grad).norm() <= 512 * 2.0 ** -24 * e.grad.norm()


def test_no_second_derivative():
    from decode_step import QKRope, rotation_tables
    cos, sin = rotation_tables(32, 64, torch.device("cuda"))
    q = torch.randn(3, 2, 64, device="cuda", requires_grad=True)
    y, _ = QKRope.apply(q, None, cos, sin, torch.arange(3, device="cuda", dtype=torch.int32), None, None, 1e-6)
    (dq,) = torch.autograd.grad(y.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.sum().backward()
