"""Refusals of the calls that serve many requests on one base model: every bad
argument is an error before anything is launched.  No kernel runs; pointers are
never followed."""
import ctypes

import pytest

import microscaling_block_quantization_amd as mx
from test_decode_abi import A, BAD_CACHES, R, cache, heads

ARG, UNSUPPORTED, ALIGN, WORKSPACE, OK = (mx.MX_ERR_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ALIGN, mx.MX_ERR_WORKSPACE, mx.MX_OK)


def read(c, k=None, v=None, tokens=4, slots=A):
    return mx.lib().mx_cache_read(R(c), slots, tokens, R(k or heads()), R(v or heads()), None)


def shared(c, q=None, out=None, batch=2, prefix=A, ahead=4, pn=A, table=A, cols=4, stride=4, lengths=A, ws=A, nbytes=1 << 40, lse=None):
    return mx.lib().mx_attend_shared(R(c), R(q or heads(n=16)), batch, prefix, ahead, pn, table, cols, stride, lengths, 1.0,
                                     R(out or heads(n=16)), lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_caches(kw, status):
    assert read(cache(**kw)) == status
    assert shared(cache(**kw)) == status


def test_read_arguments():
    assert read(cache(), tokens=-1) == ARG
    assert read(cache(), tokens=0) == OK
    assert read(cache(), slots=None) == ARG
    assert read(cache(), slots=A + 4) == ALIGN
    assert read(cache(), k=heads(n=7)) == ARG
    assert read(cache(), v=heads(dtype=0)) == ARG
    assert read(cache(), k=heads(x=None)) == ARG
    assert read(cache(), v=heads(x=A + 1)) == ALIGN
    assert read(cache(), tokens=1 << 28) == ARG
    assert mx.lib().mx_cache_read(R(cache()), A, 4, R(heads()), None, None) == ARG


def test_shared_arguments():
    assert shared(cache(), batch=0) == OK
    for bad in (dict(batch=-1), dict(cols=-1), dict(ahead=-1), dict(lengths=None), dict(pn=None), dict(table=None), dict(prefix=None),
                dict(stride=3), dict(cols=1 << 27, stride=1 << 27), dict(ahead=1 << 27), dict(q=heads(n=12), out=heads(n=12)),
                dict(out=heads(n=8)), dict(out=heads(n=16, dtype=0))):
        assert shared(cache(), **bad) == ARG, bad
    for bad in (dict(lse=A + 2), dict(lengths=A + 1), dict(table=A + 2), dict(prefix=A + 2), dict(pn=A + 2), dict(q=heads(n=16, x=A + 4))):
        assert shared(cache(), **bad) == ALIGN, bad
    c = cache(pages=4096)
    size = lambda *a: mx.lib().mx_attend_shared_workspace_size(R(c), *a)
    need = size(2, 16, 512, 512)
    assert need > 0
    for ahead, cols in ((512, 512), (512, 0), (0, 512)):
        n = size(2, 16, ahead, cols)
        assert 0 < n <= need
        at = dict(ahead=ahead, cols=cols, stride=max(cols, 1))
        assert shared(c, nbytes=n - 1, **at) == WORKSPACE
        assert shared(c, ws=None, nbytes=n, **at) == WORKSPACE
        assert shared(c, ws=A + 8, nbytes=n, **at) == ALIGN
    assert size(2, 15, 512, 512) == 0 and size(-1, 16, 512, 512) == 0 and size(2, 16, -1, 4) == 0 and size(2, 16, 4, -1) == 0


@pytest.mark.parametrize("dim,heads_,group,page", [(64, 1, 1, 16), (128, 8, 4, 16), (128, 2, 16, 64), (256, 4, 3, 1), (192, 1, 33, 24)])
def test_shared_workspace_serves_smaller_calls(dim, heads_, group, page):
    c = cache(pages=1 << 20, page=page, heads=heads_, dim=dim)
    size = lambda b, p, t: mx.lib().mx_attend_shared_workspace_size(R(c), b, heads_ * group, p, t)
    steps = [1, 2, 3, 5, 8, 13, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 256, 257, 700, 3001]
    for a, b in zip(steps, steps[1:]):
        for x, y in ((1, 1), (4, 9), (100, 7), (4000, 300)):
            assert size(a, x, y) <= size(b, x, y)
            assert size(x, a, y) <= size(x, b, y) and size(x, y, a) <= size(x, y, b)


def adapters(a=A, b=A, s=None, k=256, n=64, count=3, rank=16, dtype=1):
    return mx.MxAdapters(a, b, s, k, n, count, rank, dtype)


def lora(ad=None, x=A, tokens=4, ldx=256, ids=A, bd=1, base=A, ldb=64, yd=1, y=2 * A, ldy=64, ws=A, nbytes=1 << 40):
    return mx.lib().mx_lora(R(ad or adapters()), x, tokens, ldx, ids, bd, base, ldb, yd, y, ldy, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rank=0), UNSUPPORTED), (dict(rank=12), UNSUPPORTED), (dict(rank=264), UNSUPPORTED), (dict(k=252), UNSUPPORTED), (dict(k=0), UNSUPPORTED),
    (dict(k=-8), ARG), (dict(n=-1), ARG), (dict(count=-1), ARG), (dict(dtype=2), ARG), (dict(k=1 << 24), ARG), (dict(n=1 << 31), ARG),
])
def test_adapters(kw, status):
    assert lora(adapters(**kw), ldx=1 << 25, ldb=1 << 32, ldy=1 << 32) == status
    assert mx.lib().mx_lora_workspace_size(R(adapters(**kw)), 4) == 0


def test_lora_arguments():
    assert lora(tokens=0) == OK and lora(adapters(n=0)) == OK
    for bad in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(ldx=255), dict(ldb=63), dict(ldy=63), dict(x=None), dict(y=None),
                dict(ids=None), dict(yd=7), dict(bd=7), dict(ad=adapters(a=None)), dict(ad=adapters(b=None)),
                dict(y=A, ldy=72), dict(y=A, yd=0)):
        assert lora(**bad) == ARG, bad
    for bad in (dict(x=A + 8), dict(y=A + 8), dict(base=A + 2), dict(ids=A + 2), dict(ldx=260), dict(ad=adapters(a=A + 8)),
                dict(ad=adapters(b=A + 2)), dict(ad=adapters(s=A + 1))):
        assert lora(**bad) == ALIGN, bad
    need = mx.lib().mx_lora_workspace_size(R(adapters()), 4)
    assert need > 0 and lora(nbytes=need - 1) == WORKSPACE and lora(ws=None, nbytes=need) == WORKSPACE and lora(ws=A + 4, nbytes=need) == ALIGN
    sizes = [mx.lib().mx_lora_workspace_size(R(adapters()), t) for t in range(1, 700)]
    assert sizes == sorted(sizes)


def probs(dtype=1, z=A, tokens=4, vocab=100, ld=100, targets=A, lp=A, lse=A, h=A, top=0, tl=A, ti=A, ws=A, nbytes=1 << 40):
    return mx.lib().mx_logprobs(dtype, z, tokens, vocab, ld, targets, lp, lse, h, top, tl, ti, ws, nbytes, None)


def back(dtype=1, gl=A, gh=A, z=A, tokens=4, vocab=100, ld=100, targets=A, lse=A, h=A, dz=2 * A, ldd=100):
    return mx.lib().mx_logprobs_backward(dtype, gl, gh, z, tokens, vocab, ld, targets, lse, h, dz, ldd, None)


def test_logprobs_arguments():
    assert probs(tokens=0) == OK
    for bad in (dict(dtype=3), dict(tokens=-1), dict(vocab=0), dict(vocab=1 << 31, ld=1 << 31), dict(ld=99), dict(z=None), dict(targets=None),
                dict(lp=None), dict(lse=None), dict(h=None), dict(top=-1), dict(top=101), dict(top=5, tl=None), dict(top=5, ti=None),
                dict(tokens=1 << 31)):
        assert probs(**bad) == ARG, bad
    assert probs(top=65) == UNSUPPORTED
    for bad in (dict(z=A + 8), dict(targets=A + 4), dict(lp=A + 2), dict(lse=A + 1), dict(h=A + 2), dict(top=5, tl=A + 2), dict(top=5, ti=A + 4)):
        assert probs(**bad) == ALIGN, bad
    need = mx.lib().mx_logprobs_workspace_size(4, 200000, 20)
    big = dict(vocab=200000, ld=200000, top=20)
    assert need > 0 and probs(nbytes=need - 1, **big) == WORKSPACE and probs(ws=None, **big) == WORKSPACE and probs(ws=A + 4, **big) == ALIGN
    size = mx.lib().mx_logprobs_workspace_size
    assert size(0, 100, 5) == 0 and size(4, 100, 65) == 0 and size(4, 0, 0) == 0 and size(4, 10, 11) == 0
    for vocab in (100, 9000, 131072, 1000000):
        sizes = [size(t, vocab, 20) for t in list(range(1, 1100)) + [5000, 100000]]
        assert sizes == sorted(sizes)
    assert [size(7, v, 64) for v in (64, 8189, 8190, 10 ** 5, 10 ** 6)] == sorted(size(7, v, 64) for v in (64, 8189, 8190, 10 ** 5, 10 ** 6))


def test_logprobs_backward_arguments():
    assert back(tokens=0) == OK
    for bad in (dict(dtype=-1), dict(tokens=-1), dict(vocab=0), dict(ld=99), dict(ldd=99), dict(z=None), dict(targets=None), dict(lse=None),
                dict(dz=None), dict(h=None), dict(dz=A, ldd=108)):
        assert back(**bad) == ARG, bad
    for bad in (dict(z=A + 2), dict(dz=A + 2), dict(targets=A + 4), dict(lse=A + 2), dict(h=A + 1), dict(gl=A + 2), dict(gh=A + 2)):
        assert back(**bad) == ALIGN, bad


def test_launches_past_the_grid():
    """2^32 threads or more: refused, nothing launched (no pointer is real)."""
    c = cache(pages=1 << 20, heads=1)
    big = dict(q=heads(n=1, ts=128), out=heads(n=1, ts=128), batch=1 << 25, stride=4)
    assert shared(c, nbytes=1 << 60, **big) == ARG
    assert back(tokens=1 << 24, vocab=1 << 20, ld=1 << 20, ldd=1 << 20) == ARG
    assert probs(tokens=1 << 24, nbytes=1 << 60) == ARG


def test_struct_layouts():
    assert ctypes.sizeof(mx.MxAdapters) == 56
