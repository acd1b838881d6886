"""mx_attend_workspace_size on the host: a workspace made for the largest call
serves every smaller one (a server allocates once and sequences come and go)."""
import ctypes

import pytest

import microscaling_block_quantization_amd as mx

FORMATS = [None, mx.MXFP8_E4M3, mx.MXFP4]


def size_of(fmt, page, heads, dim, q_heads):
    f = None if fmt is None else ctypes.pointer(fmt.c())
    c = mx.MxKVCache(f, 1 << 20, 1 << 20, 1 << 20, 1 << 20, 4096, page, heads, dim)
    L = mx.lib()
    return lambda batch, cols: L.mx_attend_workspace_size(ctypes.byref(c), batch, q_heads, cols)


@pytest.mark.parametrize("fmt", FORMATS, ids=["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("page,heads,dim,group", [(16, 8, 128, 4), (16, 2, 64, 8), (24, 1, 96, 33), (64, 32, 128, 1), (16, 300, 64, 1),
                                                  (16, 4, 256, 4), (1, 3, 192, 1)])
def test_never_smaller_for_a_larger_call(fmt, page, heads, dim, group):
    size = size_of(fmt, page, heads, dim, group * heads)
    columns = sorted({0, 1, 256 // page, 256 // page + 1, 1024 // page - 1, 1024 // page, 1024 // page + 1, 4096 // page})
    batches = list(range(0, 70)) + [127, 128, 129, 255, 256, 257, 1000]
    got = [[size(b, c) for b in batches] for c in columns]
    for i in range(len(columns)):
        for j in range(len(batches)):
            assert i == 0 or got[i][j] >= got[i - 1][j], f"fewer bytes for {columns[i]} columns than for {columns[i - 1]}, batch {batches[j]}"
            assert j == 0 or got[i][j] >= got[i][j - 1], f"fewer bytes for batch {batches[j]} than for {batches[j - 1]}, {columns[i]} columns"


def test_short_tables_need_none():
    """Up to 256 tokens no batch is shared out (head dimensions up to 128)."""
    size = size_of(None, 16, 8, 128, 32)
    assert size(1000, 16) == 0 and size(1, 17) > 0
