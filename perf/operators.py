"""Cases of the decode-step operators: products of a few tokens with 4-bit
weights, the norm and rotation of query and key heads (and its gradient),
writing keys and values to a paged cache, and the attention of one new token
per sequence over that cache.

``own`` false: each operator in elementary torch operations, in 32 bits,
rounded once at the end.  ``own`` true: the framework's entry points.
``exact`` is the definition in 64 bits."""
import math

import torch

own = False
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ---- the cases -------------------------------------------------------------
def listed():
    return [
        # a small projection of one token: the launch and the latency count
        matvec("matvec int4 1x1024x1024", 1, 1024, 1024, "int4 min/max", 32, "bf16", "bf16", True),
        # the weight of the GEMM workload with the one token of a single user
        matvec("matvec mxfp4 1x14336x4096", 1, 14336, 4096, "mxfp4", 32, "bf16", "bf16", False),
        # a large layer under a small batch of users
        matvec("matvec nvfp4 16x28672x8192", 16, 28672, 8192, "nvfp4", 16, "bf16", "bf16", False),
        # one decode step of one user
        rope("rope 1 token", 1, 32, 8, 128, 128, "bf16", False),
        # a long prompt, or a training step's tokens
        rope("rope 8192 tokens", 8192, 32, 8, 128, 128, "bf16", False),
        # a short ragged training sequence, fp32, part of each head rotated
        rope("rope grad 333 tokens f32", 333, 12, 4, 96, 64, "f32", True, True),
        rope("rope grad 8192 tokens", 8192, 32, 8, 128, 128, "bf16", False, True),
        # the new tokens of a batch of users
        write("write 16 tokens bf16", 16, 8, 128, 16, "bf16"),
        # a long prompt
        write("write 8192 tokens mxfp8", 8192, 8, 128, 64, "mxfp8"),
        # one user, short context
        attend("attend 1x777 bf16", 1, 777, 32, 8, 128, 16, "bf16"),
        # a ragged batch of users
        attend("attend 32x8192 bf16", 32, 8192, 32, 8, 128, 16, "bf16"),
        # one user, long context, compressed cache
        attend("attend 1x131072 mxfp8", 1, 131072, 32, 8, 128, 64, "mxfp8"),
    ]


def matvec(name, tokens, n, k, fmt, block, x, y, bias):
    return named(name, op="matvec", tokens=tokens, n=n, k=k, fmt=fmt, block=block, x=x, y=y, bias=bias)


def rope(name, tokens, hq, hk, dim, rot, dtype, interleaved, grad=False):
    return named(name, op="rope grad" if grad else "rope", tokens=tokens, hq=hq, hk=hk, dim=dim, rot=rot, dtype=dtype,
                 interleaved=interleaved)


def write(name, tokens, hk, dim, page, cache):
    return named(name, op="write", tokens=tokens, hk=hk, dim=dim, page=page, cache=cache)


def attend(name, batch, longest, hq, hk, dim, page, cache):
    return named(name, op="attend", batch=batch, longest=longest, hq=hq, hk=hk, dim=dim, page=page, cache=cache)


def named(name, **c):
    return {"name": name, **c} if name else c


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "rope", "rope grad", "write", "attend", "attend"])
    if op == "matvec":
        fmt, block = rng.choice([("mxfp4", 32), ("nvfp4", 16), ("ue5m3", 16), ("ue5m3", 32), ("int4", 32), ("int4", 128),
                                 ("int4 min/max", 32), ("int4 min/max", 64), ("int4 min/max", 128)])
        k = -(-spread(rng, 256, 14336) // block) * block
        return matvec(None, spread(rng, 1, 16), spread(rng, 200, min(28672, 28672 * 8192 // k)), k, fmt, block,
                      rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3)
    hk = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 96, 128, 128, 256])
    if op.startswith("rope"):
        hq = hk * rng.choice([1, 3, 4, 5])
        most = 8192 * 40 * 128 // ((hq + hk) * dim * 2)
        return rope(None, spread(rng, 1, min(16384, most)), hq, hk, dim, rng.choice([dim, dim, dim // 2]),
                    rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3, op == "rope grad")
    cache = rng.choice(["bf16", "mxfp8", "mxfp4"] if op == "attend" else ["bf16", "mxfp8"])
    page = rng.choice([16, 16, 32, 64, 128, 24])
    if op == "write":
        return write(None, spread(rng, 1, 8192 * 8 * 128 // (hk * dim)), hk, dim, page, cache)
    batch = spread(rng, 1, 48)
    longest = spread(rng, 20, min(100000, 32 * 8192 * 8 * 128 // (batch * hk * dim)))
    return attend(None, batch, longest, hk * rng.choice([1, 2, 4, 5, 8, 16]), hk, dim, page, cache)


def lengths_of(c):
    """Ragged lengths: the longest first, then spread over (0, longest]; in a
    batch of four or more the last two slots hold one token and none."""
    b, n = c["batch"], c["longest"]
    got = [max(1, n - int(n * ((i * 0.618034) % 1.0) * 0.9)) for i in range(b)]
    return got if b < 4 else got[:-2] + [1, 0]


def cache_bytes(kind, values):
    return {"bf16": 2.0, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32}[kind] * values


def work(c):
    if c["op"] == "matvec":
        w = c["n"] * c["k"]
        side = 3 if c["fmt"] == "int4 min/max" else 1
        small = c["tokens"] * (c["k"] * BYTES[c["x"]] + c["n"] * BYTES[c["y"]]) + (c["n"] * BYTES[c["x"]] if c["bias"] else 0)
        return {"bytes": w / 2 + w / c["block"] * side + small, "flops": 2.0 * c["tokens"] * w}
    if c["op"] in ("rope", "rope grad"):
        values = c["tokens"] * (c["hq"] + c["hk"]) * c["dim"]
        tables = c["tokens"] * (c["rot"] * 4 + 4)
        passes = 3 if c["op"] == "rope grad" else 2
        return {"bytes": values * BYTES[c["dtype"]] * passes + tables, "flops": values * (14.0 if passes == 3 else 7.0)}
    if c["op"] == "write":
        values = 2 * c["tokens"] * c["hk"] * c["dim"]
        return {"bytes": values * 2 + cache_bytes(c["cache"], values) + 8 * c["tokens"], "flops": 3.0 * values}
    held = sum(lengths_of(c))
    small = c["batch"] * c["hq"] * (c["dim"] * 4 + 4)
    return {"bytes": cache_bytes(c["cache"], 2 * held * c["hk"] * c["dim"]) + 4 * held / c["page"] + small,
            "flops": 4.0 * held * c["hq"] * c["dim"]}


# ---- inputs ------------------------------------------------------------------
def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def pow2(e):
    """2^e in fp32 for whole e of -126 .. 127"""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def floor_log2(a):
    return torch.frexp(a)[1] - 1


def nearest_e2m1(v):
    """4-bit codes of the nearest E2M1 values"""
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return torch.bucketize(v.abs(), half).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def weights(g, c):
    """A linear layer's weight, quantized before the program serves it."""
    n, k, b = c["n"], c["k"], c["block"]
    w = (randn(g, n, k) * 0.02).view(n, k // b, b)
    amax = w.abs().amax(-1, keepdim=True)
    s = {"offsets": None, "tensor_scale": None}
    if c["fmt"] == "mxfp4":
        e = floor_log2(amax) - 2
        codes, s["scales"] = nearest_e2m1(w * pow2(-e)), (e + 127).to(torch.uint8)
    elif c["fmt"] == "nvfp4":
        t = w.abs().max().reshape(1) / (6 * 448)
        sc = (amax / 6 / t).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
        codes = nearest_e2m1(w / (sc.float() * t))
        s["scales"], s["tensor_scale"] = sc.view(torch.uint8), t
    elif c["fmt"] == "ue5m3":
        e = floor_log2(amax / 6)
        m = ((amax / 6) * pow2(-e) * 8 - 8).round().to(torch.int32)
        sc = (e + 15) * 8 + m                                       # a carry of m moves e on
        codes = nearest_e2m1(w / (pow2(sc // 8 - 15) * (1 + (sc % 8) / 8)))
        s["scales"] = sc.to(torch.uint8)
    elif c["fmt"] == "int4":
        e = floor_log2(amax) - 2
        codes, s["scales"] = (w * pow2(-e)).round().clamp(-7, 7).to(torch.int8).view(torch.uint8) & 15, (e + 127).to(torch.uint8)
    else:                                                           # int4 min/max
        off = (w.amin(-1, keepdim=True) * 1.01).to(torch.bfloat16)
        r = w.amax(-1, keepdim=True) - off.float()
        e = torch.ceil(torch.log2(r / 15)).to(torch.int32)
        codes, s["scales"] = ((w - off.float()) * pow2(-e)).round().clamp(0, 15).to(torch.uint8), (e + 127).to(torch.uint8)
        s["offsets"] = off.view(torch.int16).reshape(-1)
    s["codes"] = pack(codes.view(n, k)).contiguous()
    s["scales"] = s["scales"].view(n, k // b).contiguous()
    return s


def quantize_rows(x, kind):
    """Codes and scale codes of 1 x 32 blocks: the largest magnitude's power of
    two over the element's, values to nearest, saturated."""
    b = x.float().unflatten(-1, (-1, 32))
    e = (floor_log2(b.abs().amax(-1, keepdim=True)) - (8 if kind == "mxfp8" else 2)).clamp(-126, 127)
    v = b * pow2(-e)
    scales = (e + 127).to(torch.uint8).squeeze(-1)
    if kind == "mxfp8":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), scales
    return pack(nearest_e2m1(v).flatten(-2)), scales


def cache_of(g, kind, pages, heads, page, dim, empty=False):
    shape = (pages, heads, page, dim)
    kv = []
    for _ in range(2):
        if kind == "bf16":
            kv += [torch.zeros(shape, device=DEV, dtype=torch.bfloat16) if empty else
                   torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16), None]
        elif empty:
            kv += [torch.zeros((*shape[:3], dim // (1 if kind == "mxfp8" else 2)), device=DEV, dtype=torch.uint8),
                   torch.zeros((*shape[:3], dim // 32), device=DEV, dtype=torch.uint8)]
        else:
            kv += list(quantize_rows(torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16), kind))
    return dict(zip(("k", "k_scales", "v", "v_scales"), kv))


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "matvec":
        s |= weights(g, c)
        s["x"] = randn(g, c["tokens"], c["k"]).to(DTYPES[c["x"]])
        s["bias"] = (randn(g, c["n"]) * 0.1).to(DTYPES[c["x"]]) if c["bias"] else None
    elif c["op"] in ("rope", "rope grad"):
        t, d, dt = c["tokens"], c["dim"], DTYPES[c["dtype"]]
        rows = 16384
        angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = torch.randint(0, rows, (t,), generator=g, device=DEV, dtype=torch.int32)
        # queries and keys lie side by side, as a fused projection leaves them
        qk = randn(g, t, c["hq"] + c["hk"], d).to(dt)
        s["q"], s["k"] = qk[:, :c["hq"]], qk[:, c["hq"]:]
        s["qw"], s["kw"] = ((1 + 0.2 * randn(g, d)).to(dt) for _ in range(2))
        if c["op"] == "rope grad":
            s["dq"], s["dk"] = (1e-2 * randn(g, t, h, d).to(dt) for h in (c["hq"], c["hk"]))
    elif c["op"] == "write":
        t, page = c["tokens"], c["page"]
        pages = -(-t // page) + 8
        s |= cache_of(g, c["cache"], pages, c["hk"], page, c["dim"], True)
        s["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:t].contiguous()
        kv = randn(g, t, 2 * c["hk"], c["dim"]).to(torch.bfloat16)
        s["new_k"], s["new_v"] = kv[:, :c["hk"]], kv[:, c["hk"]:]
    else:
        page, n = c["page"], lengths_of(c)
        width = -(-c["longest"] // page)
        used = [-(-x // page) for x in n]
        pages = sum(used) + 3
        s |= cache_of(g, c["cache"], pages, c["hk"], page, c["dim"])
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(c["batch"], width, device=DEV, dtype=torch.int32)
        at = torch.arange(width, device=DEV)[None] < torch.tensor(used, device=DEV)[:, None]
        table[at] = order[: sum(used)]
        s["table"], s["lengths"] = table, torch.tensor(n, device=DEV, dtype=torch.int32)
        s["q"] = randn(g, c["batch"], c["hq"], c["dim"]).to(torch.bfloat16)
        s["scale"] = c["dim"] ** -0.5
    if own:
        handles(s)
    return s


# ---- the framework's calls ---------------------------------------------------
def handles(s):
    """The quantized weight, the cache and the workspace a program keeps."""
    import microscaling_block_quantization_amd as mx
    c = s["case"]
    s["mx"] = mx
    if c["op"] == "matvec":
        s["fmt"] = {"mxfp4": mx.Format(block_cols=c["block"]),
                    "nvfp4": mx.Format(scale=mx.SCALE_NVFP4, block_cols=c["block"]),
                    "ue5m3": mx.Format(scale=mx.SCALE_UE5M3, block_cols=c["block"]),
                    "int4": mx.Format(elem=mx.ELEM_INT4, block_cols=c["block"]),
                    "int4 min/max": mx.Format(elem=mx.ELEM_INT4, rule=mx.RULE_CEIL, asymmetric=1, block_cols=c["block"]),
                    }[c["fmt"]]
        s["w"] = mx.QTensor(c["n"], c["k"], s["codes"], s["scales"], offsets=s["offsets"], tensor_scale=s["tensor_scale"])
    if c["op"] in ("write", "attend"):
        fmt = {"bf16": None, "mxfp8": mx.MXFP8_E4M3, "mxfp4": mx.MXFP4}[c["cache"]]
        s["cache"] = mx.KVCache(fmt, s["k"], s["v"], s["k_scales"], s["v_scales"])
    if c["op"] == "attend":
        s["workspace"] = mx.alloc_attend_workspace(s["cache"], c["batch"], c["hq"], s["table"].shape[1])


def run_own(s):
    c, mx = s["case"], s["mx"]
    if c["op"] == "matvec":
        return mx.mx_matvec(s["fmt"], s["w"], s["x"], bias=s["bias"], out_dtype=DTYPES[c["y"]])
    if c["op"] == "rope":
        return mx.mx_qk_rope(s["q"], s["k"], s["cos"], s["sin"], s["positions"], s["qw"], s["kw"], eps=1e-6,
                             interleaved=c["interleaved"])
    if c["op"] == "rope grad":
        return mx.mx_qk_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["cos"], s["sin"], s["positions"], s["qw"], s["kw"],
                                      eps=1e-6, interleaved=c["interleaved"])
    if c["op"] == "write":
        mx.mx_cache_write(s["cache"], s["new_k"], s["new_v"], s["slots"])
        return written(s)
    return mx.mx_attend(s["q"], s["cache"], s["table"], s["lengths"], scale=s["scale"], lse=True, workspace=s["workspace"])


def written(s):
    """The cache after the call; 8-bit codes as the float8 values they stand for."""
    if s["case"]["cache"] == "bf16":
        return s["k"], s["v"]
    return s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn), s["k_scales"], s["v_scales"]


def run(s):
    return run_own(s) if own else run_plain(s)


# ---- plain forms, fp32 --------------------------------------------------------
def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def e2m1(codes):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return lut[codes.int()]


def e8m0(codes):
    return (codes.int() << 23).view(torch.float32)


def plain_weight(s):
    c = s["case"]
    codes = unpack(s["codes"]).view(c["n"], -1, c["block"])
    sc = s["scales"][..., None]
    if c["fmt"] == "mxfp4":
        w = e2m1(codes) * e8m0(sc)
    elif c["fmt"] == "nvfp4":
        w = e2m1(codes) * (sc.view(torch.float8_e4m3fn).float() * s["tensor_scale"])
    elif c["fmt"] == "ue5m3":
        w = e2m1(codes) * (pow2((sc.int() >> 3) - 15) * (1 + (sc & 7).float() / 8))
    elif c["fmt"] == "int4":
        w = (codes.int() - ((codes.int() & 8) << 1)).float() * e8m0(sc)
    else:
        w = s["offsets"].view(torch.bfloat16).view(c["n"], -1, 1).float() + codes.float() * e8m0(sc)
    return w.view(c["n"], c["k"])


def pairs(x, rot, interleaved):
    """The two values of each rotated pair, and what is not rotated."""
    r, rest = x[..., :rot], x[..., rot:]
    return (r[..., 0::2], r[..., 1::2], rest) if interleaved else (r[..., :rot // 2], r[..., rot // 2:], rest)


def joined(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def rotate(x, cos, sin, rot, interleaved):
    a, b, rest = pairs(x, rot, interleaved)
    return joined(a * cos - b * sin, b * cos + a * sin, rest, interleaved)


def plain_rope(s, x, w, dy=None):
    c = s["case"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    x, w = x.float(), w.float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    n = x * rstd
    if dy is None:
        return rotate(n * w, cos, sin, c["rot"], c["interleaved"]).to(DTYPES[c["dtype"]])
    g = rotate(dy.float(), cos, -sin, c["rot"], c["interleaved"])
    h = g * w
    dx = rstd * (h - n * (h * n).mean(-1, keepdim=True))
    return dx.to(DTYPES[c["dtype"]]), (g * n).sum((0, 1))


def plain_rows(values, scales, kind):
    if kind == "bf16":
        return values.float()
    v = values.view(torch.float8_e4m3fn).float() if kind == "mxfp8" else e2m1(unpack(values))
    return (v.unflatten(-1, (-1, 32)) * e8m0(scales)[..., None]).flatten(-2)


def plain_attend(s):
    c = s["case"]
    b, hk, d = c["batch"], c["hk"], c["dim"]
    at = s["table"].long()
    side = [plain_rows(s[n][at], None if s[n + "_scales"] is None else s[n + "_scales"][at], c["cache"]) for n in ("k", "v")]
    k, v = (x.transpose(1, 2).reshape(b, hk, -1, d) for x in side)
    q = s["q"].float().view(b, hk, -1, d)
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * s["scale"]
    dead = torch.arange(score.shape[-1], device=DEV)[None] >= s["lengths"][:, None]
    score = score.masked_fill(dead[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).squeeze(-1)
    return o.view(b, -1, d).to(torch.bfloat16), torch.where(total.squeeze(-1) == 0, -math.inf, lse).view(b, -1)


def run_plain(s):
    c = s["case"]
    if c["op"] == "matvec":
        y = torch.matmul(s["x"].float(), plain_weight(s).t())
        return (y if s["bias"] is None else y + s["bias"].float()).to(DTYPES[c["y"]])
    if c["op"] == "rope":
        return plain_rope(s, s["q"], s["qw"]), plain_rope(s, s["k"], s["kw"])
    if c["op"] == "rope grad":
        dq, dqw = plain_rope(s, s["q"], s["qw"], s["dq"])
        dk, dkw = plain_rope(s, s["k"], s["kw"], s["dk"])
        return dq, dk, dqw, dkw
    if c["op"] == "write":
        page, off = s["slots"] // c["page"], s["slots"] % c["page"]
        if c["cache"] == "bf16":
            s["k"][page, :, off], s["v"][page, :, off] = s["new_k"], s["new_v"]
        else:
            s["k"][page, :, off], s["k_scales"][page, :, off] = quantize_rows(s["new_k"], c["cache"])
            s["v"][page, :, off], s["v_scales"][page, :, off] = quantize_rows(s["new_v"], c["cache"])
        return written(s)
    return plain_attend(s)


# ---- the definitions in 64 bits -------------------------------------------------
def value64(codes, bits, man, bias):
    """The value of a sign-magnitude minifloat code."""
    codes = codes.long()
    mag = codes & ((1 << (bits - 1)) - 1)
    e, m = mag >> man, (mag & ((1 << man) - 1)).double() / (1 << man)
    v = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((e - bias).double()))
    return torch.where((codes >> (bits - 1)) & 1 == 1, -v, v)


def scale64(codes):
    return torch.ldexp(torch.ones_like(codes, dtype=torch.float64), codes.int() - 127)


def nibbles(codes):
    out = codes.new_empty((*codes.shape[:-1], 2 * codes.shape[-1]))
    out[..., 0::2], out[..., 1::2] = codes % 16, codes // 16
    return out


def exact_matvec(s):
    c = s["case"]
    y = torch.empty(c["tokens"], c["n"], device=DEV, dtype=torch.float64)
    for r in range(0, c["n"], 4096):
        part = slice(r, min(c["n"], r + 4096))
        codes = nibbles(s["codes"][part])
        sc = s["scales"][part].repeat_interleave(c["block"], 1)
        if c["fmt"] == "mxfp4":
            w = value64(codes, 4, 1, 1) * scale64(sc)
        elif c["fmt"] in ("nvfp4", "ue5m3"):
            w = value64(codes, 4, 1, 1) * value64(sc, 9, 3, 7 if c["fmt"] == "nvfp4" else 15)
        elif c["fmt"] == "int4":
            w = torch.where(codes > 7, codes.double() - 16, codes.double()) * scale64(sc)
        else:
            off = s["offsets"].view(torch.bfloat16).view(c["n"], -1)[part].double()
            w = off.repeat_interleave(c["block"], 1) + codes.double() * scale64(sc)
        y[:, part] = torch.mm(s["x"].double(), w.t().contiguous())
    y = y if s["tensor_scale"] is None else y * s["tensor_scale"].double()
    return y if s["bias"] is None else y + s["bias"].double()


def exact_rope(s, x, w, dy=None):
    """Each pair as one complex number times e^(i angle)."""
    c = s["case"]
    i = s["positions"].long()
    turn = torch.complex(s["cos"].double()[i], s["sin"].double()[i])[:, None]
    x, w = x.double(), w.double()
    rstd = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def turned(v, by):
        v = v.clone()
        first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, c["rot"] // 2)
        second = slice(1, c["rot"], 2) if c["interleaved"] else slice(c["rot"] // 2, c["rot"])
        z = torch.complex(v[..., first].contiguous(), v[..., second].contiguous()) * by
        v[..., first], v[..., second] = z.real, z.imag
        return v

    if dy is None:
        return turned(x * rstd * w, turn)
    g = turned(dy.double(), turn.conj())
    dw = (g * x * rstd).sum((0, 1))
    g = g * w
    return rstd * g - x * rstd ** 3 * (g * x).sum(-1, keepdim=True) / c["dim"], dw


def exact_write(s):
    c = s["case"]
    got = []
    for name in ("k", "v"):
        rows = s["new_" + name].double()
        if c["cache"] == "mxfp8":
            b = rows.unflatten(-1, (-1, 32))
            b = b / torch.exp2(torch.floor(torch.log2(b.abs().amax(-1, keepdim=True))) - 8)
            step = torch.exp2(torch.floor(torch.log2(b.abs().clamp(min=2.0 ** -6))) - 3)
            rows = (torch.round(b / step) * step).clamp(-448, 448).flatten(-2)
        full = torch.zeros(s[name].shape[0], c["page"], c["hk"], c["dim"], device=DEV, dtype=torch.float64)
        full.view(-1, c["hk"], c["dim"])[s["slots"]] = rows
        got.append(full.transpose(1, 2).contiguous())
    return tuple(got) if c["cache"] == "bf16" else (*got, None, None)


def exact_attend(s):
    c = s["case"]
    o = torch.zeros(c["batch"], c["hq"], c["dim"], device=DEV, dtype=torch.float64)
    lse = torch.full((c["batch"], c["hq"]), -math.inf, device=DEV, dtype=torch.float64)

    def rows(name, pages, h, n):
        x = s[name][pages, h].flatten(0, 1)[:n]
        if c["cache"] == "bf16":
            return x.double()
        v = value64(x, 8, 3, 7) if c["cache"] == "mxfp8" else value64(nibbles(x), 4, 1, 1)
        return v * scale64(s[name + "_scales"][pages, h].flatten(0, 1)[:n]).repeat_interleave(32, 1)

    for b, n in enumerate(lengths_of(c)):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // c["page"])].long()
        for h in range(c["hk"]):
            own_heads = slice(h * c["hq"] // c["hk"], (h + 1) * c["hq"] // c["hk"])
            z = torch.mm(rows("k", pages, h, n), s["q"][b, own_heads].double().t().contiguous()) * s["scale"]
            lse[b, own_heads] = torch.logsumexp(z, 0)
            o[b, own_heads] = torch.mm(torch.softmax(z, 0).t().contiguous(), rows("v", pages, h, n))
    return o, lse


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "matvec":
        return exact_matvec(s)
    if c["op"] == "rope":
        return exact_rope(s, s["q"], s["qw"]), exact_rope(s, s["k"], s["kw"])
    if c["op"] == "rope grad":
        dq, dqw = exact_rope(s, s["q"], s["qw"], s["dq"])
        dk, dkw = exact_rope(s, s["k"], s["kw"], s["dk"])
        return dq, dk, dqw, dkw
    return exact_write(s) if c["op"] == "write" else exact_attend(s)
