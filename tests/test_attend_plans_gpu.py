"""Ways a call of the attention is split, at the sizes where one gives way to
another.  Checks and tolerances are those of test_attend_gpu."""
import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_attend_gpu import build, check_attend

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_one_workspace_for_a_server():
    """Allocated for 32 sequences of up to 1024 tokens, which need none, then
    used by as many and by fewer, which share out their tokens."""
    page, hk, dim = 16, 8, 128
    rng = np.random.default_rng(1)
    lengths = [int(v) for v in rng.integers(1, 1000, 32)]
    lengths[3], lengths[7], lengths[31] = 0, 1024, 1
    cache, table, n = build("bf16", lengths, hk, dim, page, extra_cols=0)
    assert table.shape[1] == 64
    ws = mx.alloc_attend_workspace(cache, 32, 32, 64).fill_(0xFF)
    assert ws.numel() > 0
    q = torch.randn(32, 32, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(BF16)
    for batch in (32, 31, 16, 9, 1):
        out, lse = mx.mx_attend(q[:batch], cache, table[:batch], n[:batch], lse=True, workspace=ws)
        check_attend(cache, table[:batch], n[:batch], q[:batch], dim ** -0.5, out, lse, f"batch {batch}")
