"""Products with 4-bit weights at the ends of their scales' range, against
float64.  The tolerance is test_matvec_gpu's: operands are exact, so an fp32
output is off by at most (K + 64) 2^-23 of the sum of |terms|, terms being
|q s x| and |o x| with INT4's u s and 8 s taken as 16 s.  Macro scales give
INT4 operands more bits: they lie on a grid of 2^-129 (bf16's smallest step,
2^-133, over the 2^-4 that INT4 operands carry), half of which times |x| is
added per weight."""
import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx

pytestmark = pytest.mark.gpu
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def nibbles(codes):
    out = np.empty((codes.shape[0], codes.shape[1] * 2), np.int64)
    out[:, 0::2], out[:, 1::2] = codes & 15, codes >> 4
    return out


def values(elem, asym, codes):
    n = nibbles(codes)
    if elem == mx.ELEM_E2M1:
        return E2M1[n]
    return (n if asym else np.where(n > 7, n - 16, n)).astype(np.float64)


def bf16(a):
    t = torch.from_numpy(np.clip(a, -3e38, 3e38)).float().to(torch.bfloat16)
    return t, t.double().numpy()


def check(fmt, w, val, big, rows, x, grid=0.0, label=""):
    y = mx.mx_matvec(fmt, w, x, out_dtype=torch.float32).double().cpu().numpy()[:, rows]
    x64 = x.double().cpu().numpy()
    want = x64 @ val[rows].T
    tol = (val.shape[1] + 64) * 2.0 ** -23 * (np.abs(x64) @ big[rows].T) + grid * np.abs(x64).sum(1, keepdims=True)
    err = np.abs(y - want)
    assert (err <= tol).all(), f"{label}: {np.nanmax(err / tol):.2f} of the tolerance, NaN {np.isnan(y).sum()}"


@pytest.mark.parametrize("elem,asym", [(mx.ELEM_E2M1, 0), (mx.ELEM_E2M1, 1), (mx.ELEM_INT4, 0), (mx.ELEM_INT4, 1)])
@pytest.mark.parametrize("block", [8, 16, 32, 64])
@pytest.mark.parametrize("k", [256, 4224])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_e8m0_scale(elem, asym, block, k, dtype):
    """A row for each scale code (up to where the largest value still is
    finite), its neighbours in some blocks."""
    rng = np.random.default_rng(block + k)
    top = {mx.ELEM_E2M1: 252, mx.ELEM_INT4: 254 if asym == 0 else 250}[elem]
    n = top + 1
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    sc = np.clip(np.arange(n)[:, None] - rng.integers(0, 3, (n, k // block)), 0, 254).astype(np.uint8)
    if elem == mx.ELEM_INT4 and not asym:
        # -8 .. 7 times 2^125 and more is not finite throughout: there -1 .. 0 alone
        codes[252:] = np.where(rng.random((n - 252, k // 2)) < 0.5, 0xFF, 0x00)
    s = np.repeat(2.0 ** (sc.astype(np.float64) - 127), block, 1)
    val = values(elem, asym, codes) * s
    big = np.abs(val) + (16 * s if elem == mx.ELEM_INT4 else 0)
    off = None
    if asym:
        off, o = bf16(rng.standard_normal((n, k // block)) * 8 * 2.0 ** (sc.astype(np.float64) - 127))
        o = np.repeat(o, block, 1)
        val, big = val + o, big + 2 * np.abs(o)
        off = off.view(torch.int16).cuda()
    w = mx.QTensor(n, k, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda(), offsets=off)
    fmt = mx.Format(elem=elem, asymmetric=asym, rule=mx.RULE_CEIL, block_cols=block)
    x = torch.from_numpy(rng.standard_normal((3, k)))
    half = np.arange(n) < 127
    check(fmt, w, val, big, half, (x * 2.0 ** 60).to(dtype).cuda(), label="small scales")
    check(fmt, w, val, big, ~half, (x * 2.0 ** -60).to(dtype).cuda(), label="large scales")


@pytest.mark.parametrize("elem", [mx.ELEM_E2M1, mx.ELEM_INT4])
@pytest.mark.parametrize("k", [256, 4224])
def test_smallest_scales_with_macro_scales(elem, k):
    rng = np.random.default_rng(k)
    n = 40
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    sc = np.repeat(np.arange(n, dtype=np.uint8)[:, None] // 4, k // 32, 1)
    mac = rng.integers(56, 64, (n, k // 128), dtype=np.uint8)                    # UE4M3 1 .. 1.875
    s = np.repeat(2.0 ** (sc.astype(np.float64) - 127), 32, 1) * np.repeat(1 + (mac - 56) / 8, 128, 1)
    val = values(elem, 0, codes) * s
    big = np.abs(val) + (16 * s if elem == mx.ELEM_INT4 else 0)
    w = mx.QTensor(n, k, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda(), macro_scales=torch.from_numpy(mac).cuda())
    x = (torch.from_numpy(rng.standard_normal((3, k))) * 2.0 ** 60).to(torch.bfloat16).cuda()
    grid = 2.0 ** -130 if elem == mx.ELEM_INT4 else 0.0
    check(mx.Format(elem=elem, macro_cols=128), w, val, big, np.arange(n) >= 0, x, grid)


def test_small_int4_weights_of_a_tensor():
    """Weights of 2^-127 .. 2^-118 and given offsets: 3 x 2^-127 is not 0."""
    k, x = 256, torch.full((1, 256), 2.0 ** 100, device="cuda", dtype=torch.bfloat16)
    codes, sc = torch.full((16, k // 2), 0x33, device="cuda", dtype=torch.uint8), torch.zeros(16, k // 32, device="cuda", dtype=torch.uint8)
    y = mx.mx_matvec(mx.Format(elem=mx.ELEM_INT4), mx.QTensor(16, k, codes, sc), x, out_dtype=torch.float32)
    assert (y == 3 * k * 2.0 ** -27).all()
    off = torch.full((16, k // 32), 2.0 ** -120 + 2.0 ** -127, device="cuda").to(torch.bfloat16).view(torch.int16)
    f = mx.Format(elem=mx.ELEM_INT4, asymmetric=1, rule=mx.RULE_CEIL)
    y = mx.mx_matvec(f, mx.QTensor(16, k, codes, sc, offsets=off), x, out_dtype=torch.float32)
    assert (y == k * (2.0 ** -20 + 2.0 ** -27 + 3 * 2.0 ** -27)).all()
