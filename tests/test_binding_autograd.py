"""The decode-step calls and autograd: a tensor that a call writes into counts
as changed in place, so a backward that saved it says so instead of using what
it has become.  No GPU: see on_host."""
import pytest
import torch

import microscaling_block_quantization_amd as mx
from on_host import Machine, gpu

BF16 = torch.bfloat16


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def heads(t, h, d=64):
    return gpu(torch.zeros(t, h, d, dtype=BF16))


def args():
    return (gpu(torch.zeros(40, 32)), gpu(torch.zeros(40, 32)), gpu(torch.zeros(3, dtype=torch.int32)),
            gpu(torch.zeros(64, dtype=BF16)), gpu(torch.zeros(64, dtype=BF16)))


def cache():
    return mx.KVCache(None, *(gpu(torch.zeros(80, 2, 16, 64, dtype=BF16)) for _ in range(2)))


def weight():
    return mx.QTensor(64, 256, gpu(torch.zeros(8192, dtype=torch.uint8)), gpu(torch.zeros(512, dtype=torch.uint8)))


def versions(*ts):
    return [t._version for t in ts]


def test_outputs_given_count_as_changed(machine):
    q, k = heads(3, 4), heads(3, 2)
    mx.mx_qk_rope(q, k, *args(), q_out=q, k_out=k)
    assert versions(q, k) == [1, 1]
    gq, gk, dq = heads(3, 4), heads(3, 2), heads(3, 4)
    mx.mx_qk_rope_backward(gq, gk, q, k, *args(), dq=dq, dk=gk)
    assert versions(gq, dq, gk, q, k) == [0, 1, 1, 1, 1]
    y, x = gpu(torch.zeros(2, 64)), gpu(torch.zeros(2, 256))
    mx.mx_matvec(mx.MXFP4, weight(), x, y=y)
    out, lse = heads(2, 4), gpu(torch.zeros(2, 4))
    table, n = gpu(torch.zeros(2, 30, dtype=torch.int32)), gpu(torch.zeros(2, dtype=torch.int32))
    a = heads(2, 4)
    mx.mx_attend(a, cache(), table, n, out=out, lse=lse)
    assert versions(y, x, out, lse, a, table, n) == [1, 0, 1, 1, 0, 0, 0]


def test_new_outputs_and_inference_tensors(machine):
    q, k = mx.mx_qk_rope(heads(3, 4), heads(3, 2), *args())
    assert versions(q, k) == [0, 0]
    with torch.inference_mode():
        h = heads(3, 4)
        mx.mx_qk_rope(h, None, *args()[:3], q_out=h)
    mx.mx_qk_rope(h, None, *args()[:3], q_out=h)          # has no counter
    assert len(machine.launches) == 3


def test_a_backward_that_saved_the_heads_notices(machine):
    """y = q^2 keeps q; q turned in place before the backward."""
    leaf = torch.ones(3, 4, 64, dtype=BF16, requires_grad=True)
    q = (leaf * 2).as_subclass(type(heads(1, 1)))
    y = (q * q).sum()
    with torch.no_grad():
        mx.mx_qk_rope(q, None, *args()[:3], q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
