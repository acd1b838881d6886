"""The largest launches of the adapters' two products: a call either of whose grids
would hold 2^32 threads or more is refused before anything is launched, and the
sizes just below are not.  Pointers are never followed: refused calls launch
nothing, and the others run only where there is no GPU to launch on."""
import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_requests_abi import adapters, lora

below = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that hold nothing")

# up to 16 tokens: 256 threads for 64 outputs; above: 256 for 256 outputs and a
# run of up to 64 tiles of 16 tokens
WIDE = [(16, (1 << 30) - 63, (1 << 30) - 64), (1, (1 << 30) - 63, (1 << 30) - 64), (1 << 24, 1 << 18, (1 << 18) - 256)]


def call(tokens, n, dtype):
    return lora(adapters(n=n, rank=8, dtype=dtype), tokens=tokens, ldb=n, ldy=n, bd=0, yd=1)


@pytest.mark.parametrize("tokens,n,_", WIDE)
@pytest.mark.parametrize("dtype", [0, 1])
def test_refused(tokens, n, _, dtype):
    assert call(tokens, n, dtype) == mx.MX_ERR_ARG


@below
@pytest.mark.parametrize("tokens,_,n", WIDE)
@pytest.mark.parametrize("dtype", [0, 1])
def test_below(tokens, _, n, dtype):
    assert call(tokens, n, dtype) == mx.MX_ERR_HIP
