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


@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 24])
def test_whole_sequences_of_many_tiles(kind, dtype, page):
    """Enough sequences of up to 1024 tokens that each is one workgroup's: its
    eight waves take up to four tiles of 32 each, with empty sequences, of one
    token, and around the tiles' and the waves' ends."""
    hk, dim = 8, 128
    rng = np.random.default_rng(page)
    lengths = [0, 1, 31, 32, 33, 255, 256, 257, 288, 289, 511, 512, 513, 777, 1000, 1008, 0]
    lengths += [int(v) for v in rng.integers(1, 1008, 23)]
    cache, table, n = build(kind, lengths, hk, dim, page, extra_cols=0)
    assert 256 < table.shape[1] * page <= 1024 and len(lengths) * hk >= 256
    q = torch.randn(len(lengths), 2 * hk, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(dtype)
    # a call that is not shared out takes no workspace
    empty = torch.empty(0, device="cuda", dtype=torch.uint8)
    out, lse = mx.mx_attend(q, cache, table, n, lse=True, workspace=empty)
    check_attend(cache, table, n, q, dim ** -0.5, out, lse, f"{kind} {dtype} page {page}")


@pytest.mark.parametrize("dim,group", [(64, 16), (96, 3), (128, 17)])
def test_whole_sequences_of_other_heads(dim, group):
    """The same with peaked scores (maxima that grow from tile to tile), other
    head dimensions and head tiles that are part full."""
    hk, page = 2, 32
    rng = np.random.default_rng(dim)
    lengths = [int(v) for v in rng.integers(0, 900, 128)]
    cache, table, n = build("mxfp8", lengths, hk, dim, page, extra_cols=0, spread=20.0)
    assert 256 < table.shape[1] * page <= 1024
    q = torch.randn(128, group * hk, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).to(BF16)
    out, lse = mx.mx_attend(q, cache, table, n, lse=True, workspace=torch.empty(0, device="cuda", dtype=torch.uint8))
    some = [0, 1, 2, 63, 127, int(n.argmax()), int(n.argmin())]
    check_attend(cache, table[some], n[some], q[some], dim ** -0.5, out[some], lse[some], f"{dim} {group}")


@pytest.mark.parametrize("dim", [128, 256])
def test_wide_head_tiles_in_a_graph(dim):
    """16 query heads of a key-value head take over 64 KiB of LDS, which a
    launch asks for; captured, every replay (its query renewed) is the eager
    call's, bit for bit."""
    lengths = [200, 0, 77]
    cache, table, n = build("bf16", lengths, 2, dim, 16)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(3, 32, dim, device="cuda", generator=g).to(BF16)
    ws = mx.alloc_attend_workspace(cache, 3, 32, table.shape[1])
    held = q.clone()
    mx.mx_attend(held, cache, table, n, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = mx.mx_attend(held, cache, table, n, lse=True, workspace=ws)
    for i in range(6):
        held.copy_(torch.randn(3, 32, dim, device="cuda", generator=g))
        ws.fill_(0xFF)
        graph.replay()
        want, wl = mx.mx_attend(held, cache, table, n, lse=True)
        if i % 3 == 0:
            torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl), f"replay {i}"
    check_attend(cache, table, n, held, dim ** -0.5, out, lse, f"{dim}")
