"""Products of a few tokens with a 4-bit weight (mx_matvec) against float64
products of the oracle's dequantized weights.

Tolerances.  W's values enter exactly and fp32 x as an exact sum, so an fp32
output is a sum of K products (and K / b offset terms) in fp32: off by at most
(K + 64) u S with u = 2^-23 per step (twice the rounding of an addition, so
truncating adders are covered) and S the sum of |terms|, terms being |q s x|
and |o x| (INT4 symmetric: q = 0 .. 15 and o = -8 s).  A bf16 output adds half
a unit in its last place, 2^-8 of its magnitude."""
import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx
import oracle

pytestmark = pytest.mark.gpu

FORMATS = {
    "mxfp4": dict(),
    "mxfp4 b8": dict(block_cols=8),
    "mxfp4 b16 ceil": dict(block_cols=16, rule=1),
    "mxfp4 b256": dict(block_cols=256),
    "mbs 1x16": dict(block_cols=16, macro_cols=128),
    "mbs 1x32": dict(block_cols=32, macro_cols=128),
    "nvfp4": dict(scale=2, block_cols=16),
    "ue4m3 b32": dict(scale=1, block_cols=32),
    "ue5m3 b8": dict(scale=3, block_cols=8),
    "e2m1 asym": dict(asymmetric=1, rule=1),
    "e2m1 asym b16": dict(asymmetric=1, rule=1, block_cols=16),
    "int4": dict(elem=1),
    "int4 b8": dict(elem=1, block_cols=8),
    "int4 b128": dict(elem=1, block_cols=128),
    "int4 ue4m3 b16": dict(elem=1, scale=1, block_cols=16),
    "int4 nvfp4 b32": dict(elem=1, scale=2, block_cols=32),
    "int4 mbs b16": dict(elem=1, macro_cols=128, block_cols=16),
    "int4 asym": dict(elem=1, asymmetric=1, rule=1),
    "int4 asym b16": dict(elem=1, asymmetric=1, rule=1, block_cols=16),
    "int4 asym b64": dict(elem=1, asymmetric=1, rule=1, block_cols=64),
}


def quantized(rng, n, k, kw):
    """A weight of uneven rows, quantized by the oracle, as a device QTensor,
    with its values and the magnitudes its terms can reach, in float64."""
    w = (rng.standard_normal((n, k)) * 0.02 * np.exp(rng.uniform(-3, 3, (n, 1)))).astype(np.float32)
    r = oracle.quantize(w, oracle.Format(**kw))
    dev = lambda a: None if a is None else torch.from_numpy(a.reshape(-1).copy()).cuda()
    q = mx.QTensor(n, k, dev(r["codes"]), dev(r["scales"]),
                   offsets=None if r["offsets"] is None else dev(r["offsets"].view(np.int16)),
                   macro_scales=dev(r["macro_scales"]), tensor_scale=dev(r["tensor_scale"]))
    val = r["dequant"].astype(np.float64)
    big = np.abs(val)
    b = kw.get("block_cols", 32)
    if kw.get("asymmetric"):
        off = np.repeat(np.abs(oracle.bf16_bits_to_f32(r["offsets"])), b, 1)
        big = big + 2 * off
    elif kw.get("elem") == 1:
        # q s with q up to 15 and 8 s: the block's largest magnitude is at least 4 s
        peak = np.repeat(np.abs(val).reshape(n, k // b, b).max(-1), b, 1)
        big = big + 4 * peak
    return q, val, big


def tokens(rng, t, k, dtype, pad=0):
    x = torch.from_numpy(rng.standard_normal((t, k + pad)).astype(np.float32)).to(dtype).cuda()
    return x[:, :k]


def check(y, x, val, big, bias=None, label=""):
    x64 = x.double().cpu().numpy()
    want = x64 @ val.T
    tol = (val.shape[1] + 64) * 2.0 ** -23 * (np.abs(x64) @ big.T)
    if bias is not None:
        b = bias.double().cpu().numpy()
        want = want + b
        tol = tol + 2.0 ** -23 * (np.abs(b) + np.abs(want))
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{label}: {np.max(err / np.maximum(tol, 1e-300)):.2f} of the tolerance"


@pytest.mark.parametrize("name", FORMATS)
@pytest.mark.parametrize("x_dtype,y_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                            (torch.float32, torch.float32)])
def test_formats(name, x_dtype, y_dtype):
    kw = FORMATS[name]
    rng = np.random.default_rng(len(name) * 7 + 1)
    for t, n, k in ((1, 33, 256), (3, 48, 1280), (16, 17, 2304), (5, 100, 4352)):
        print(name, t, n, k, x_dtype, y_dtype, flush=True)
        q, val, big = quantized(rng, n, k, kw)
        x = tokens(rng, t, k, x_dtype)
        check(mx.mx_matvec(mx.Format(**kw), q, x, out_dtype=y_dtype), x, val, big, label=f"{t}x{n}x{k}")


@pytest.mark.parametrize("name,step", [("mxfp4", 32), ("mxfp4 b8", 8), ("nvfp4", 16), ("ue5m3 b8", 8), ("int4 b8", 8),
                                       ("int4", 32), ("int4 asym b16", 16), ("mbs 1x16", 128)])
def test_odd_lengths(name, step):
    """K that ends inside a lane's 32 codes, a 128-wide step, or a stage."""
    kw = FORMATS[name]
    rng = np.random.default_rng(5)
    for k in (step, 3 * step, 128 + step, 9 * 128 - step, 1024 + step, 8192 + 5 * step):
        if k % step or k % 8:
            continue
        for t, n in ((1, 1), (2, 15), (16, 16), (7, 37)):
            print(name, t, n, k, flush=True)
            q, val, big = quantized(rng, n, k, kw)
            x = tokens(rng, t, k, torch.bfloat16)
            check(mx.mx_matvec(mx.Format(**kw), q, x, out_dtype=torch.float32), x, val, big, label=f"{t}x{n}x{k}")


@pytest.mark.parametrize("t", [2, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens_strides_and_bias(t, dtype):
    """Token counts around the tile, strided x and y (whose gaps stay untouched), a bias."""
    rng = np.random.default_rng(t)
    n, k, pad = 75, 672, 40
    for name in ("mxfp4", "int4 asym", "nvfp4"):
        kw = FORMATS[name]
        q, val, big = quantized(rng, n, k, kw)
        x = tokens(rng, t, k, dtype, pad)
        bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dtype).cuda()
        full = torch.full((t, n + 13), 7.0, device="cuda", dtype=dtype)
        y = mx.mx_matvec(mx.Format(**kw), q, x, bias=bias, y=full[:, :n])
        check(y, x, val, big, bias, label=name)
        assert (full[:, n:] == 7).all(), "wrote past the row"


@pytest.mark.parametrize("elem,scale", [(0, 0), (0, 1), (0, 3), (1, 0), (1, 1)])
def test_exact_small_integers(elem, scale):
    """Unit scales and small whole tokens: every partial sum is exact in fp32."""
    rng = np.random.default_rng(9)
    n, k = 50, 1536
    unit = {0: 127, 1: 7 << 3, 3: 15 << 3}[scale]
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    sc = np.full((n, k // 32), unit, np.uint8)
    val = oracle.dequantize(oracle.Format(elem=elem, scale=scale), {"codes": codes, "scales": sc}, n, k).astype(np.float64)
    q = mx.QTensor(n, k, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.from_numpy(rng.integers(-4, 5, (6, k)).astype(np.float32)).to(dtype).cuda()
        y = mx.mx_matvec(mx.Format(elem=elem, scale=scale), q, x, out_dtype=torch.float32)
        assert np.array_equal(y.double().cpu().numpy(), x.double().cpu().numpy() @ val.T)


@pytest.mark.parametrize("elem", [0, 1])
def test_extreme_scales(elem):
    """E8M0 scales far from one, each row its own: 2^-100 .. 2^100."""
    rng = np.random.default_rng(10)
    n, k = 41, 256
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    sc = np.repeat(np.arange(27, 27 + 5 * n, 5, dtype=np.uint8)[:, None], k // 32, 1)
    val = oracle.dequantize(oracle.Format(elem=elem), {"codes": codes, "scales": sc}, n, k).astype(np.float64)
    big = np.abs(val) + (16 * 2.0 ** (sc[:, :1].astype(np.float64) - 127) if elem else 0)
    q = mx.QTensor(n, k, torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
    x = tokens(rng, 4, k, torch.bfloat16)
    check(mx.mx_matvec(mx.Format(elem=elem), q, x, out_dtype=torch.float32), x, val, big)


def test_wide_fp32_tokens():
    """fp32 tokens whose low bits matter and whose magnitudes span 2^-60 .. 2^60."""
    rng = np.random.default_rng(12)
    q, val, big = quantized(rng, 20, 512, FORMATS["mxfp4"])
    x = torch.from_numpy((rng.standard_normal((5, 512)) * 2.0 ** rng.integers(-60, 60, (5, 1))).astype(np.float32)).cuda()
    check(mx.mx_matvec(mx.MXFP4, q, x), x, val, big)


@pytest.mark.parametrize("name", ["mxfp4", "nvfp4", "ue5m3 b8", "int4", "int4 asym", "int4 ue4m3 b16", "mbs 1x16"])
def test_nan_scale_marks_its_row(name):
    kw = FORMATS[name]
    rng = np.random.default_rng(13)
    q, val, big = quantized(rng, 40, 512, kw)
    bad = {0: 0xFF, 1: 0x7F, 2: 0x7F, 3: 0xFF}[kw.get("scale", 0)]
    per = 512 // kw.get("block_cols", 32)
    q.scales.view(40, per)[7, per - 1] = bad
    q.scales.view(40, per)[39, 0] = bad
    x = tokens(rng, 3, 512, torch.bfloat16)
    y = mx.mx_matvec(mx.Format(**kw), q, x, out_dtype=torch.float32)
    assert y[:, [7, 39]].isnan().all()
    ok = [i for i in range(40) if i not in (7, 39)]
    check(y[:, ok], x, val[ok], big[ok])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_bad_token_stays_alone(dtype, what):
    rng = np.random.default_rng(14)
    for name in ("mxfp4", "int4", "nvfp4"):
        q, val, big = quantized(rng, 64, 544, FORMATS[name])
        x = tokens(rng, 9, 544, dtype).clone()
        x[4, 333] = what
        y = mx.mx_matvec(mx.Format(**FORMATS[name]), q, x, out_dtype=torch.float32)
        hit = torch.from_numpy(val[:, 333] != 0)
        assert (~y[4].cpu().isfinite())[hit].all()
        ok = [i for i in range(9) if i != 4]
        check(y[ok], x[ok], val, big, label=name)


def test_nothing_to_do_and_same_bits():
    rng = np.random.default_rng(15)
    q, _, _ = quantized(rng, 64, 4096, FORMATS["nvfp4"])
    f = mx.Format(**FORMATS["nvfp4"])
    assert mx.mx_matvec(f, q, torch.empty((0, 4096), dtype=torch.bfloat16, device="cuda")).shape == (0, 64)
    x = tokens(rng, 11, 4096, torch.bfloat16)
    first = mx.mx_matvec(f, q, x, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(mx.mx_matvec(f, q, x, out_dtype=torch.float32), first)


@pytest.mark.parametrize("name,t,n,k,x_dtype", [("mxfp4", 2, 4100, 4096, torch.bfloat16), ("nvfp4", 16, 8200, 4640, torch.bfloat16),
                                                ("int4 asym b64", 3, 4200, 9216, torch.bfloat16), ("int4 asym", 1, 40005, 1024, torch.float32),
                                                ("mxfp4", 5, 33000, 2048, torch.float32), ("int4 b128", 9, 12400, 4096, torch.bfloat16),
                                                ("mbs 1x16", 4, 9000, 4224, torch.bfloat16)])
def test_many_rows(name, t, n, k, x_dtype):
    """Workgroups of several row tiles, the last one part full, and several
    passes over K, on random codes and scales."""
    kw = FORMATS[name]
    rng = np.random.default_rng(n)
    b = kw.get("block_cols", 32)
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    lo = {0: 118, 1: 40, 2: 40, 3: 100}[kw.get("scale", 0)]
    sc = rng.integers(lo, lo + 16, (n, k // b), dtype=np.uint8)
    off = oracle.f32_to_bf16_bits(rng.standard_normal((n, k // b)).astype(np.float32)) if kw.get("asymmetric") else None
    mac = rng.integers(56, 65, (n, k // 128), dtype=np.uint8) if kw.get("macro_cols") else None      # 1 .. 2
    ts = np.array([0.037], np.float32) if kw.get("scale") == 2 else None
    val = oracle.dequantize(oracle.Format(**kw), {"codes": codes, "scales": sc, "offsets": off, "macro_scales": mac,
                                                  "tensor_scale": ts}, n, k)
    dev = lambda a: None if a is None else torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()
    q = mx.QTensor(n, k, dev(codes), dev(sc), offsets=dev(off), macro_scales=dev(mac), tensor_scale=dev(ts))
    x = tokens(rng, t, k, x_dtype)
    y = mx.mx_matvec(mx.Format(**kw), q, x, out_dtype=torch.float32)
    w = torch.from_numpy(val).cuda().double()
    big = w.abs()
    if kw.get("asymmetric"):
        big += 2 * torch.from_numpy(np.abs(oracle.bf16_bits_to_f32(off))).cuda().double().repeat_interleave(b, 1)
    elif kw.get("elem") == 1:
        big += 16 * torch.ldexp(torch.ones(sc.shape, device="cuda", dtype=torch.float64),
                                dev(sc).int() - 127).repeat_interleave(b, 1)
    want = torch.mm(x.double(), w.t().contiguous())
    tol = (k + 64) * 2.0 ** -23 * torch.mm(x.double().abs(), big.t().contiguous())
    err = (y.double() - want).abs()
    assert (err <= tol).all(), f"{(err / tol).max().item():.2f} of the tolerance"
