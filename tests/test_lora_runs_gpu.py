"""Adapters over prompts so long that a workgroup of the second product goes down
several tiles of tokens with an adapter's weights held, against float64 with the
tolerance of test_lora_gpu."""
import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_lora_gpu import BF16, F32, check, make

pytestmark = pytest.mark.gpu


def prompts(tokens, count, seed):
    """Ids in stretches of one to 200 tokens, an adapter, another, none, the same
    again after a gap, and a stretch of single tokens of any."""
    g = torch.Generator().manual_seed(seed)
    n = tokens // 20 + 200
    long = torch.randint(1, 200, (n,), generator=g)
    long = torch.where(torch.rand(n, generator=g) < 0.3, 16 * (1 + long // 16), long)             # whole tiles among them
    ids = torch.repeat_interleave(torch.randint(-1, count, (n,), generator=g), long)[:tokens]
    ids[tokens // 2:tokens // 2 + 300] = torch.randint(-1, count + 1, (300,), generator=g)        # count: no such adapter
    ids[tokens // 4:tokens // 4 + 1600] = 1                                                       # longer than a workgroup's run
    return ids.to(torch.int32).cuda()


# tokens, outputs: runs of 3, 4 and 12 tiles
@pytest.mark.parametrize("tokens,n", [(25003, 1000), (65537, 500), (45000, 2049)])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 72, 256])
@pytest.mark.parametrize("dtype,base,out", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, BF16, F32)])
def test_runs_of_tiles(tokens, n, rank, dtype, base, out):
    print(tokens, n, rank, dtype, base, out, flush=True)
    ad, x, _, b = make(tokens, n, 64, rank, 5, dtype, base)
    ids = prompts(tokens, 5, rank)
    y = mx.mx_lora(x, ad, ids, b, out_dtype=out)
    for at in range(0, tokens, 8192):
        rows = slice(at, at + 8192)
        check(ad, x[rows], ids[rows], b[rows], y[rows], f"tokens from {at}")


@pytest.mark.parametrize("rank,dtype", [(16, BF16), (16, F32), (72, BF16)])
def test_longest_runs(rank, dtype):
    """131072 tokens of 16400 outputs: 65 groups of outputs, 64 tiles a run; rows
    from all over it."""
    tokens, n = 131072, 16400
    ad, x, _, _ = make(tokens, n, 8, rank, 5, dtype, None)
    ids = prompts(tokens, 5, rank)
    y = mx.mx_lora(x, ad, ids, None, out_dtype=BF16)
    for at in (0, tokens // 4 - 100, tokens // 2 - 100, 100000, tokens - 1100):
        rows = slice(at, at + 1100)
        check(ad, x[rows], ids[rows], None, y[rows], f"tokens from {at}")
