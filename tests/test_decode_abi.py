"""Refusals of the decode-step entry points: every bad argument is an error
before anything is launched.  No kernel runs; pointers are never followed."""
import ctypes

import pytest

import microscaling_block_quantization_amd as mx

A = 1 << 20                      # an aligned address that is never followed
R = ctypes.byref


def matvec(kw=None, rows=64, cols=256, xd=1, x=A, tokens=1, ldx=256, bias=None, y=A, ldy=64, yd=1, **q):
    f = mx.Format(**(kw or {})).c()
    t = mx.MxQTensor(q.get("codes", A), q.get("scales", A), q.get("offsets"), q.get("macro"), q.get("ts"), None, rows, cols)
    return mx.lib().mx_matvec(R(f), R(t), xd, x, tokens, ldx, bias, y, ldy, yd, None)


@pytest.mark.parametrize("kw,args,status", [
    (dict(elem=2), {}, mx.MX_ERR_UNSUPPORTED), (dict(elem=5), {}, mx.MX_ERR_UNSUPPORTED), (dict(elem=4), {}, mx.MX_ERR_UNSUPPORTED),
    (dict(scale=4, rule=1), {}, mx.MX_ERR_UNSUPPORTED), (dict(hadamard=32), {}, mx.MX_ERR_UNSUPPORTED),
    (dict(block_rows=32, block_cols=1), {}, mx.MX_ERR_UNSUPPORTED), (dict(block_rows=32, block_cols=32), {}, mx.MX_ERR_UNSUPPORTED),
    (dict(block_cols=24), {}, mx.MX_ERR_ARG), ({}, dict(cols=250, ldx=256), mx.MX_ERR_ARG),
    ({}, dict(xd=2), mx.MX_ERR_ARG), ({}, dict(yd=-1), mx.MX_ERR_ARG), ({}, dict(tokens=-1), mx.MX_ERR_ARG),
    ({}, dict(ldx=255), mx.MX_ERR_ARG), ({}, dict(ldy=63), mx.MX_ERR_ARG), ({}, dict(rows=-1), mx.MX_ERR_ARG),
    ({}, dict(x=None), mx.MX_ERR_ARG), ({}, dict(y=None), mx.MX_ERR_ARG), ({}, dict(codes=None), mx.MX_ERR_ARG),
    ({}, dict(scales=None), mx.MX_ERR_ARG), (dict(elem=1, asymmetric=1), {}, mx.MX_ERR_ARG),
    (dict(macro_cols=128), {}, mx.MX_ERR_ARG), (dict(scale=2, block_cols=16), {}, mx.MX_ERR_ARG),
    ({}, dict(x=A + 8), mx.MX_ERR_ALIGN), ({}, dict(y=A + 2), mx.MX_ERR_ALIGN), ({}, dict(bias=A + 4), mx.MX_ERR_ALIGN),
    ({}, dict(codes=A + 4), mx.MX_ERR_ALIGN), ({}, dict(ldx=260), mx.MX_ERR_ALIGN),
    ({}, dict(cols=0, ldx=8), mx.MX_ERR_UNSUPPORTED), ({}, dict(tokens=1048561), mx.MX_ERR_ARG),
    ({}, dict(cols=1 << 24, ldx=1 << 24), mx.MX_ERR_ARG),
    ({}, dict(tokens=0), mx.MX_OK), ({}, dict(rows=0), mx.MX_OK),
])
def test_matvec(kw, args, status):
    assert matvec(kw, **args) == status


def rope(**kw):
    a = dict(tokens=4, dim=128, rot=128, inter=0, wd=1, qw=A, kw=A, cos=A, sin=A, rows=100, pos=A, eps=1e-6)
    a.update(kw)
    return mx.MxRope(a["tokens"], a["dim"], a["rot"], a["inter"], a["wd"], a["qw"], a["kw"], a["cos"], a["sin"], a["rows"],
                     a["pos"], a["eps"])


def heads(x=A, ts=1024, hs=128, n=8, dtype=1):
    return mx.MxHeads(x, ts, hs, n, dtype)


def call_rope(r, q=None, k=None, qo=None, ko=None):
    q, k, qo, ko = (h or heads() for h in (q, k, qo, ko))
    return mx.lib().mx_qk_rope(R(r), R(q), R(k), R(qo), R(ko), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), mx.MX_ERR_ARG), (dict(dim=100), mx.MX_ERR_UNSUPPORTED), (dict(dim=0), mx.MX_ERR_UNSUPPORTED),
    (dict(dim=1032), mx.MX_ERR_UNSUPPORTED), (dict(rot=130), mx.MX_ERR_ARG), (dict(rot=3), mx.MX_ERR_ARG),
    (dict(rot=-2), mx.MX_ERR_ARG), (dict(inter=2), mx.MX_ERR_ARG), (dict(wd=9), mx.MX_ERR_ARG),
    (dict(eps=-1.0), mx.MX_ERR_ARG), (dict(eps=float("nan")), mx.MX_ERR_ARG), (dict(cos=None), mx.MX_ERR_ARG),
    (dict(pos=None), mx.MX_ERR_ARG), (dict(rows=0), mx.MX_ERR_ARG), (dict(qw=A + 2), mx.MX_ERR_ALIGN),
    (dict(sin=A + 4), mx.MX_ERR_ALIGN), (dict(pos=A + 2), mx.MX_ERR_ALIGN), (dict(tokens=1 << 28), mx.MX_ERR_ARG), (dict(tokens=0), mx.MX_OK),
])
def test_rope_description(kw, status):
    assert call_rope(rope(**kw)) == status
    g = heads()
    rc = mx.lib().mx_qk_rope_backward(R(rope(**kw)), R(g), R(g), R(g), R(g), R(g), R(g), A, A, None, 0, None)
    assert rc == (status if status != mx.MX_OK else mx.MX_ERR_WORKSPACE)


@pytest.mark.parametrize("bad,status", [
    (heads(x=None), mx.MX_ERR_ARG), (heads(n=0), mx.MX_ERR_ARG), (heads(dtype=0), mx.MX_ERR_ARG), (heads(dtype=3), mx.MX_ERR_ARG),
    (heads(n=7), mx.MX_ERR_ARG), (heads(x=A + 2), mx.MX_ERR_ALIGN), (heads(ts=1028), mx.MX_ERR_ALIGN),
    (heads(hs=129), mx.MX_ERR_ALIGN),
])
def test_rope_heads(bad, status):
    for which in ("q", "k", "qo", "ko"):
        assert call_rope(rope(), **{which: bad}) == status, which


def test_rope_partners():
    L, g = mx.lib(), heads()
    assert L.mx_qk_rope(R(rope()), R(g), R(g), R(g), None, None) == mx.MX_ERR_ARG
    assert L.mx_qk_rope(R(rope()), None, R(g), R(g), R(g), None) == mx.MX_ERR_ARG
    back = lambda r, *a: L.mx_qk_rope_backward(R(r), *a, None)
    need = L.mx_qk_rope_workspace_size(R(rope()))
    assert need > 0 and L.mx_qk_rope_workspace_size(R(rope(qw=None, kw=None))) == 0
    six = [R(g)] * 6
    assert back(rope(), *six, None, A, A, need) == mx.MX_ERR_ARG          # a weight without its gradient
    assert back(rope(kw=None), *six, A, A, A, need) == mx.MX_ERR_ARG      # and the other way round
    assert back(rope(), *six, A, A, A, need - 1) == mx.MX_ERR_WORKSPACE
    assert back(rope(), *six, A, A, None, need) == mx.MX_ERR_WORKSPACE
    assert back(rope(), *six, A, A, A + 8, need) == mx.MX_ERR_ALIGN
    assert back(rope(), R(g), None, R(g), R(g), R(g), R(g), A, A, A, need) == mx.MX_ERR_ARG


def cache(fmt=None, k=A, v=A, ks=A, vs=A, pages=10, page=16, heads=8, dim=128):
    return mx.MxKVCache(None if fmt is None else ctypes.pointer(mx.Format(**fmt).c()), k, v, ks, vs, pages, page, heads, dim)


BAD_CACHES = [
    (dict(dim=80), mx.MX_ERR_UNSUPPORTED), (dict(dim=512), mx.MX_ERR_UNSUPPORTED), (dict(page=0), mx.MX_ERR_ARG),
    (dict(page=65537), mx.MX_ERR_ARG), (dict(heads=0), mx.MX_ERR_ARG), (dict(pages=-1), mx.MX_ERR_ARG),
    (dict(pages=0), mx.MX_ERR_ARG), (dict(pages=1 << 40), mx.MX_ERR_ARG), (dict(k=None), mx.MX_ERR_ARG), (dict(v=None), mx.MX_ERR_ARG),
    (dict(fmt={}, ks=None), mx.MX_ERR_ARG), (dict(k=A + 8), mx.MX_ERR_ALIGN), (dict(fmt={}, vs=A + 4), mx.MX_ERR_ALIGN),
    (dict(fmt=dict(elem=1)), mx.MX_ERR_UNSUPPORTED), (dict(fmt=dict(elem=6)), mx.MX_ERR_UNSUPPORTED),
    (dict(fmt=dict(scale=1)), mx.MX_ERR_UNSUPPORTED), (dict(fmt=dict(block_cols=16)), mx.MX_ERR_UNSUPPORTED),
    (dict(fmt=dict(round=1)), mx.MX_ERR_UNSUPPORTED), (dict(fmt=dict(hadamard=32)), mx.MX_ERR_UNSUPPORTED),
    (dict(fmt=dict(asymmetric=1)), mx.MX_ERR_UNSUPPORTED), (dict(fmt=dict(rule=2, oas_tau=1.0)), mx.MX_ERR_ARG),
]


def write(c, k=None, v=None, tokens=4, slots=A):
    return mx.lib().mx_cache_write(R(c), R(k or heads()), R(v or heads()), tokens, slots, None)


def attend(c, q=None, out=None, batch=2, table=A, cols=4, stride=4, lengths=A, ws=A, nbytes=1 << 40, lse=None):
    return mx.lib().mx_attend(R(c), R(q or heads(n=16)), batch, table, cols, stride, lengths, 1.0, R(out or heads(n=16)), lse, ws,
                              nbytes, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_caches(kw, status):
    assert write(cache(**kw)) == status
    assert attend(cache(**kw)) == status


def test_write_arguments():
    assert write(cache(), tokens=-1) == mx.MX_ERR_ARG
    assert write(cache(), tokens=0) == mx.MX_OK
    assert write(cache(), slots=None) == mx.MX_ERR_ARG
    assert write(cache(), slots=A + 4) == mx.MX_ERR_ALIGN
    assert write(cache(), k=heads(n=7)) == mx.MX_ERR_ARG
    assert write(cache(), v=heads(dtype=0)) == mx.MX_ERR_ARG
    assert write(cache(), v=heads(x=A + 1)) == mx.MX_ERR_ALIGN
    assert write(cache(), tokens=1 << 28) == mx.MX_ERR_ARG


def test_attend_arguments():
    assert attend(cache(), batch=0) == mx.MX_OK
    for bad in (dict(batch=-1), dict(cols=-1), dict(lengths=None), dict(table=None), dict(stride=3), dict(cols=1 << 27, stride=1 << 27),
                dict(q=heads(n=12), out=heads(n=12)), dict(out=heads(n=8)), dict(out=heads(n=16, dtype=0))):
        assert attend(cache(), **bad) == mx.MX_ERR_ARG, bad
    for bad in (dict(lse=A + 2), dict(lengths=A + 1), dict(table=A + 2)):
        assert attend(cache(), **bad) == mx.MX_ERR_ALIGN, bad
    assert attend(cache(), q=heads(n=16, x=A + 4)) == mx.MX_ERR_ALIGN
    c = cache(pages=4096)
    need = mx.lib().mx_attend_workspace_size(R(c), 2, 16, 512)
    assert need > 0
    assert attend(c, cols=512, stride=512, nbytes=need - 1) == mx.MX_ERR_WORKSPACE
    assert attend(c, cols=512, stride=512, ws=None, nbytes=need) == mx.MX_ERR_WORKSPACE
    assert attend(c, cols=512, stride=512, ws=A + 8, nbytes=need) == mx.MX_ERR_ALIGN
    assert mx.lib().mx_attend_workspace_size(R(c), 2, 15, 512) == 0
    assert mx.lib().mx_attend_workspace_size(R(c), 0, 16, 512) == 0
    assert mx.lib().mx_attend_workspace_size(R(c), 2, 16, 0) == 0


def test_struct_layouts():
    assert ctypes.sizeof(mx.MxHeads) == 32 and ctypes.sizeof(mx.MxRope) == 80 and ctypes.sizeof(mx.MxKVCache) == 64
