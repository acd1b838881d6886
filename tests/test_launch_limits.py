"""The largest launches: sizes whose grid would hold 2^32 threads or more are
refused before anything is launched, and the sizes just below are not.  Pointers
are never followed: refused calls launch nothing, and the others run only where
there is no GPU to launch on."""
import ctypes

import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_decode_abi import A, R, attend, cache, call_rope, heads, matvec, rope, write

below = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that hold nothing")

# what is just too large, what is just small enough
MATVEC = [(dict(rows=(1 << 28) - 31, cols=8, ldx=8, ldy=1 << 30), dict(block_cols=8)),
          (dict(rows=(1 << 30) - 127, cols=4096, ldx=4096, ldy=1 << 30), {})]


@pytest.mark.parametrize("args,fmt", MATVEC)
def test_matvec(args, fmt):
    assert matvec(fmt, **args) == mx.MX_ERR_ARG
    assert matvec(fmt, **(args | dict(tokens=20))) == mx.MX_ERR_ARG


@below
@pytest.mark.parametrize("args,fmt", MATVEC)
def test_matvec_below(args, fmt):
    assert matvec(fmt, **(args | dict(rows=args["rows"] - 1))) == mx.MX_ERR_HIP


# one head of `dim` values: lanes of 16 values, a power of two of them, at least 4
ROPE = [(64, 1 << 30), (128, 1 << 29), (80, 1 << 29), (1024, 1 << 26)]


def rope_of(dim, tokens, dtype=1):
    h = heads(ts=dim, hs=dim, n=1, dtype=dtype)
    p = R(h)
    return mx.lib().mx_qk_rope(R(rope(dim=dim, rot=0, tokens=tokens, kw=None)), p, None, p, None, None)


@pytest.mark.parametrize("dim,tokens", ROPE)
@pytest.mark.parametrize("dtype", [0, 1])
def test_rope(dim, tokens, dtype):
    assert rope_of(dim, tokens, dtype) == mx.MX_ERR_ARG


@below
@pytest.mark.parametrize("dim,tokens", ROPE)
def test_rope_below(dim, tokens):
    assert rope_of(dim, tokens - 256) == mx.MX_ERR_HIP


# lanes of 8 values; 256 threads hold as many whole vectors as fit
WRITE = [(256, 8), (192, 10), (128, 16), (96, 21), (64, 32)]


def write_of(dim, tokens):
    h = heads(ts=dim, hs=dim, n=1)
    return write(cache(heads=1, dim=dim), k=h, v=h, tokens=tokens)


@pytest.mark.parametrize("dim,per", WRITE)
def test_cache_write(dim, per):
    assert write_of(dim, ((1 << 24) - 1) * per + 1) == mx.MX_ERR_ARG


@below
@pytest.mark.parametrize("dim,per", WRITE)
def test_cache_write_below(dim, per):
    assert write_of(dim, ((1 << 24) - 1) * per) == mx.MX_ERR_HIP


# batch x query heads: the join's 256 threads for each; whole sequences' 512 for
# each key-value head and 16 query heads
ATTEND = [(dict(heads=1), 1, 100, 1 << 24), (dict(heads=1), 1, 4, 1 << 23), (dict(heads=8), 8, 4, 1 << 20), (dict(heads=1), 16, 4, 1 << 23)]


def attend_of(c, q_heads, cols, batch):
    h = heads(n=q_heads)
    return attend(cache(**c), q=h, out=h, batch=batch, cols=cols, stride=cols, nbytes=1 << 62)


@pytest.mark.parametrize("c,q_heads,cols,batch", ATTEND)
def test_attend(c, q_heads, cols, batch):
    assert attend_of(c, q_heads, cols, batch) == mx.MX_ERR_ARG


@below
@pytest.mark.parametrize("c,q_heads,cols,batch", ATTEND)
def test_attend_below(c, q_heads, cols, batch):
    assert attend_of(c, q_heads, cols, batch - 1) == mx.MX_ERR_HIP


@below
def test_what_the_header_promises():
    """Sizes it says always run."""
    assert matvec(dict(block_cols=8), rows=(1 << 28) - 32, cols=8, ldx=8, ldy=1 << 30) == mx.MX_ERR_HIP
    assert rope_of(1024, (1 << 26) - 256) == mx.MX_ERR_HIP
    assert write_of(256, (1 << 27) - 8) == mx.MX_ERR_HIP
    assert attend_of(dict(heads=1), 1, 4, (1 << 23) - 1) == mx.MX_ERR_HIP
