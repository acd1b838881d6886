"""Cases of the operators that serve many requests on one quantized base model:
the attention of a batch whose sequences share a long prefix, the prefix's
cached keys and values read back, low-rank adapters of many requests beside a
shared projection, and the log probabilities of given tokens with entropy and
top alternatives, with their gradient.

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
        # a few users behind one short instruction
        shared("shared 4x40 on 777 bf16", 4, 777, 40, 32, 8, 128, 16, "bf16", "bf16"),
        # a ragged batch of users behind one long instruction
        shared("shared 32x512 on 8192 bf16", 32, 8192, 512, 32, 8, 128, 16, "bf16", "bf16"),
        # many questions about one long document, compressed cache
        shared("shared 64x1024 on 32768 mxfp8", 64, 32768, 1024, 32, 8, 128, 64, "mxfp8", "bf16"),
        # a short prefix handed to another cache
        read("read 300 tokens mxfp4", 300, 4, 64, 16, "mxfp4", "f32"),
        # a long document's keys and values for the products of its next chunk
        read("read 65536 tokens mxfp8", 65536, 8, 128, 64, "mxfp8", "bf16"),
        # one user's token at a small projection: launches and latency count
        lora("lora 1x1024x1024 rank 8", 1, 1024, 1024, 8, 4, False, "bf16", "bf16", "bf16"),
        # a decode step of many users, each with an adapter of their own, at a
        # large projection whose product is still fp32
        lora("lora 16x14336x4096 rank 16", 16, 14336, 4096, 16, 32, False, "bf16", "f32", "bf16"),
        # prompts of eight users
        lora("lora 8192x14336x4096 rank 16", 8192, 14336, 4096, 16, 8, True, "bf16", "bf16", "bf16"),
        # one user's next token
        logprobs("logprobs 1x32000 f32 top 20", 1, 32000, 20, "f32", False),
        # the next tokens of a batch of users
        logprobs("logprobs 64x131072 bf16 top 20", 64, 131072, 20, "bf16", True),
        # a short ragged training sequence, a vocabulary of odd size
        logprobs("logprobs grad 333x50001 f32", 333, 50001, 0, "f32", False, True),
        # a training step's tokens
        logprobs("logprobs grad 4096x131072 bf16", 4096, 131072, 0, "bf16", False, True),
    ]


def shared(name, batch, prefix, longest, hq, hk, dim, page, cache, dtype):
    return named(name, op="shared", batch=batch, prefix=prefix, longest=longest, hq=hq, hk=hk, dim=dim, page=page, cache=cache,
                 dtype=dtype)


def read(name, tokens, hk, dim, page, cache, dtype):
    return named(name, op="read", tokens=tokens, hk=hk, dim=dim, page=page, cache=cache, dtype=dtype)


def lora(name, tokens, n, k, rank, adapters, prompt, x, base, y):
    return named(name, op="lora", tokens=tokens, n=n, k=k, rank=rank, adapters=adapters, prompt=prompt, x=x, base=base, y=y)


def logprobs(name, tokens, vocab, top, dtype, masked, grad=False):
    return named(name, op="logprobs grad" if grad else "logprobs", tokens=tokens, vocab=vocab, top=top, dtype=dtype, masked=masked)


def named(name, **c):
    return {"name": name, **c} if name else c


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "read", "lora", "lora", "logprobs", "logprobs", "logprobs grad"])
    if op in ("shared", "read"):
        hk = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 96, 128, 128, 256])
        cache = rng.choice(["bf16", "mxfp8", "mxfp4"])
        page = rng.choice([16, 16, 32, 64, 128, 24])
        if op == "read":
            return read(None, spread(rng, 1, 65536 * 8 * 128 // (2 * hk * dim)), hk, dim, page, cache, rng.choice(["bf16", "bf16", "f32"]))
        hq = hk * rng.choice([1, 2, 4, 4, 8, 16])
        batch = spread(rng, 1, 96)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = 64 * 32768 * 32 * 128 // (batch * hq * dim * (4 if dtype == "f32" else 1))
        prefix = spread(rng, 30, min(100000, most))
        longest = spread(rng, 1, min(2048, prefix, max(1, 64 * 1024 * 8 * 128 // (2 * batch * hk * dim))))
        return shared(None, batch, prefix, longest, hq, hk, dim, page, cache, dtype)
    if op == "lora":
        k, rank = 8 * spread(rng, 32, 1792), rng.choice([8, 16, 16, 32, 64])
        prompt = rng.random() < 0.4
        tokens = spread(rng, 20, 4000) if prompt else spread(rng, 1, 48)
        n = spread(rng, 200, min(28672, 8192 * 14336 // tokens // 2))
        return lora(None, tokens, n, k, rank, spread(rng, 1, 40), prompt, rng.choice(["bf16", "bf16", "f32"]),
                    rng.choice(["bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]))
    vocab = spread(rng, 1000, 160000)
    dtype = rng.choice(["bf16", "f32"])
    if op == "logprobs":
        top = rng.choice([0, 1, 5, 20, 32])
        return logprobs(None, spread(rng, 1, 512 if top else min(4096, 4096 * 131072 // (vocab * 2))), vocab, top, dtype, rng.random() < 0.3)
    return logprobs(None, spread(rng, 1, min(4096, 4096 * 131072 // (vocab * 2))), vocab, 0, dtype, rng.random() < 0.3, True)


def lengths_of(c):
    """Ragged lengths: the longest first, then spread over (0, longest]; in a
    batch of four or more the last two slots hold one token and none."""
    b, n = c["batch"], c["longest"]
    got = [max(1, n - int(n * ((i * 0.618034) % 1.0) * 0.9)) for i in range(b)]
    return got if b < 4 else got[:-2] + [1, 0]


def cache_bytes(kind, values):
    return {"bf16": 2.0, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32}[kind] * values


def work(c):
    if c["op"] == "shared":
        held = c["prefix"] + sum(lengths_of(c))
        small = c["batch"] * c["hq"] * (c["dim"] * 2 * BYTES[c["dtype"]] + 4)
        return {"bytes": cache_bytes(c["cache"], 2 * held * c["hk"] * c["dim"]) + 4 * held / c["page"] + small,
                "flops": 4.0 * c["hq"] * c["dim"] * (c["batch"] * c["prefix"] + sum(lengths_of(c)))}
    if c["op"] == "read":
        values = 2 * c["tokens"] * c["hk"] * c["dim"]
        return {"bytes": cache_bytes(c["cache"], values) + BYTES[c["dtype"]] * values + 8 * c["tokens"], "flops": 1.0 * values}
    if c["op"] == "lora":
        used = min(c["adapters"], c["tokens"])
        rows = c["tokens"] * (c["k"] * BYTES[c["x"]] + c["n"] * (BYTES[c["base"]] + BYTES[c["y"]]) + 4)
        return {"bytes": rows + used * (c["k"] + c["n"]) * c["rank"] * BYTES[c["x"]], "flops": 2.0 * c["tokens"] * c["rank"] * (c["k"] + c["n"])}
    values = c["tokens"] * c["vocab"]
    if c["op"] == "logprobs":
        return {"bytes": values * BYTES[c["dtype"]] + c["tokens"] * (20 + 12 * c["top"]), "flops": 6.0 * values}
    return {"bytes": 2 * values * BYTES[c["dtype"]] + c["tokens"] * 24, "flops": 8.0 * values}


# ---- inputs ------------------------------------------------------------------
def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def pow2(e):
    """2^e in fp32 for whole e of -126 .. 127"""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def nearest_e2m1(v):
    """4-bit codes of the nearest E2M1 values"""
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return torch.bucketize(v.abs(), half).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)


def quantize_rows(x, kind):
    """Codes and scale codes of 1 x 32 blocks: the largest magnitude's power of
    two over the element's, values to nearest, saturated."""
    b = x.float().unflatten(-1, (-1, 32))
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 1 - (8 if kind == "mxfp8" else 2)).clamp(-126, 127)
    v = b * pow2(-e)
    scales = (e + 127).to(torch.uint8).squeeze(-1)
    if kind == "mxfp8":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), scales
    codes = nearest_e2m1(v).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales


def cache_of(g, kind, pages, heads, page, dim):
    shape = (pages, heads, page, dim)
    kv = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        kv += [x, None] if kind == "bf16" else list(quantize_rows(x, kind))
    return dict(zip(("k", "k_scales", "v", "v_scales"), kv))


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "shared":
        page, n = c["page"], lengths_of(c)
        ahead = -(-c["prefix"] // page)
        used = [-(-x // page) for x in n]
        pages = ahead + sum(used) + 3
        s |= cache_of(g, c["cache"], pages, c["hk"], page, c["dim"])
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["prefix"], order = order[:ahead].contiguous(), order[ahead:]
        s["prefix_length"] = torch.tensor([c["prefix"]], device=DEV, dtype=torch.int32)
        table = torch.zeros(c["batch"], -(-c["longest"] // page), device=DEV, dtype=torch.int32)
        at = torch.arange(table.shape[1], device=DEV)[None] < torch.tensor(used, device=DEV)[:, None]
        table[at] = order[: sum(used)]
        s["table"], s["lengths"] = table, torch.tensor(n, device=DEV, dtype=torch.int32)
        s["q"] = randn(g, c["batch"], c["hq"], c["dim"]).to(DTYPES[c["dtype"]])
        s["scale"] = c["dim"] ** -0.5
    elif c["op"] == "read":
        page = c["page"]
        need = -(-c["tokens"] // page)
        s |= cache_of(g, c["cache"], need + 5, c["hk"], page, c["dim"])
        order = torch.randperm(need + 5, generator=g, device=DEV)[:need]
        s["slots"] = (order[:, None] * page + torch.arange(page, device=DEV)).view(-1)[: c["tokens"]].contiguous()
    elif c["op"] == "lora":
        dt, t, a = DTYPES[c["x"]], c["tokens"], c["adapters"]
        s["x"] = randn(g, t, c["k"]).to(dt)
        s["a"] = (randn(g, a, c["rank"], c["k"]) * c["k"] ** -0.5).to(dt)
        s["b"] = (randn(g, a, c["n"], c["rank"]) * 0.1).to(dt)
        s["scales"] = torch.rand(a, generator=g, device=DEV) + 0.5
        s["base"] = randn(g, t, c["n"]).to(DTYPES[c["base"]])
        # a request in eight has no adapter; a prompt's tokens lie together
        of = torch.randint(0, a, (t,), generator=g, device=DEV)
        if c["prompt"]:
            of = torch.sort(of).values
            order = torch.randperm(a, generator=g, device=DEV)
            s["ids"] = torch.where(order[of] % 8 == 7, -1, order[of]).to(torch.int32)
        else:
            s["ids"] = torch.where(torch.rand(t, generator=g, device=DEV) < 0.125, -1, of).to(torch.int32)
    else:
        t, v = c["tokens"], c["vocab"]
        z = randn(g, t, v) * 2.5
        # a model's likeliest tokens stand out
        z.scatter_add_(1, torch.randint(0, v, (t, 8), generator=g, device=DEV), randn(g, t, 8).abs() * 5)
        target = torch.randint(0, v, (t,), generator=g, device=DEV)
        target = torch.where(torch.rand(t, generator=g, device=DEV) < 0.7, z.argmax(1), target)
        if c["masked"]:                                             # what a grammar or a padded vocabulary rules out
            out = (torch.rand(v, generator=g, device=DEV) < 0.4)[None] & (torch.arange(v, device=DEV)[None] != target[:, None])
            z.masked_fill_(out, -math.inf)
        s["logits"], s["target"] = z.to(DTYPES[c["dtype"]]), target
        if c["op"] == "logprobs grad":
            s["d_logprob"], s["d_entropy"] = randn(g, t) / t, randn(g, t) * 0.01 / t
            zf = s["logits"].float()
            s["lse"] = torch.logsumexp(zf, 1)
            lp = zf - s["lse"][:, None]
            s["entropy"] = -(lp.exp() * lp.clamp(min=-1e30)).sum(1)
    if own:
        handles(s)
    return s


# ---- the framework's calls ---------------------------------------------------
def handles(s):
    """The cache, the adapters and the workspaces a program keeps."""
    import microscaling_block_quantization_amd as mx
    c = s["case"]
    s["mx"] = mx
    if c["op"] in ("shared", "read"):
        fmt = {"bf16": None, "mxfp8": mx.MXFP8_E4M3, "mxfp4": mx.MXFP4}[c["cache"]]
        s["cache"] = mx.KVCache(fmt, s["k"], s["v"], s["k_scales"], s["v_scales"])
    if c["op"] == "shared":
        s["workspace"] = mx.alloc_attend_shared_workspace(s["cache"], c["batch"], c["hq"], s["prefix"].shape[0], s["table"].shape[1])
    elif c["op"] == "lora":
        s["adapters"] = mx.Adapters(s["a"], s["b"], s["scales"])
        s["workspace"] = mx.alloc_lora_workspace(s["adapters"], c["tokens"])
    elif c["op"] == "logprobs":
        s["workspace"] = mx.alloc_logprobs_workspace(c["tokens"], c["vocab"], c["top"])


def run_own(s):
    c, mx = s["case"], s["mx"]
    if c["op"] == "shared":
        return mx.mx_attend_shared(s["q"], s["cache"], s["prefix"], s["prefix_length"], s["table"], s["lengths"], scale=s["scale"],
                                   lse=True, workspace=s["workspace"])
    if c["op"] == "read":
        return mx.mx_cache_read(s["cache"], s["slots"], out_dtype=DTYPES[c["dtype"]])
    if c["op"] == "lora":
        return mx.mx_lora(s["x"], s["adapters"], s["ids"], s["base"], out_dtype=DTYPES[c["y"]], workspace=s["workspace"])
    if c["op"] == "logprobs":
        return mx.mx_logprobs(s["logits"], s["target"], top=c["top"], workspace=s["workspace"])
    return mx.mx_logprobs_backward(s["d_logprob"], s["d_entropy"], s["logits"], s["target"], s["lse"], s["entropy"])


def run(s):
    return run_own(s) if own else run_plain(s)


# ---- plain forms, fp32 --------------------------------------------------------
def plain_rows(values, scales, kind):
    if kind == "bf16":
        return values.float()
    if kind == "mxfp8":
        v = values.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=values.device)
        v = lut[torch.stack((values & 15, values >> 4), -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 32)) * (scales.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def plain_side(s, name, at):
    """Rows of the pages `at`, heads first: ... x heads x tokens x dim."""
    x = plain_rows(s[name][at], None if s[name + "_scales"] is None else s[name + "_scales"][at], s["case"]["cache"])
    return x.transpose(-4, -3).flatten(-3, -2)


def plain_shared(s):
    c = s["case"]
    b, hk, d = c["batch"], c["hk"], c["dim"]
    q = s["q"].float().view(b, hk, -1, d)
    kp, vp = (plain_side(s, n, s["prefix"].long()) for n in ("k", "v"))
    ko, vo = (plain_side(s, n, s["table"].long()) for n in ("k", "v"))
    qp = q.transpose(0, 1).reshape(hk, -1, d)                       # all sequences' heads beside each other
    zp = torch.matmul(qp, kp.transpose(-1, -2).contiguous()) * s["scale"]
    zp = zp.masked_fill(torch.arange(zp.shape[-1], device=DEV) >= s["prefix_length"], -math.inf)
    zo = torch.matmul(q, ko.transpose(-1, -2).contiguous()) * s["scale"]
    dead = torch.arange(zo.shape[-1], device=DEV)[None] >= s["lengths"][:, None]
    zo = zo.masked_fill(dead[:, None, None], -math.inf)
    over = lambda x: x.view(hk, b, -1, x.shape[-1]).transpose(0, 1)
    m = torch.maximum(over(zp.amax(-1, keepdim=True)), zo.amax(-1, keepdim=True))
    m = torch.where(m == -math.inf, 0.0, m)
    pp = torch.exp(zp - m.transpose(0, 1).reshape(hk, -1, 1))
    po = torch.exp(zo - m)
    total = over(pp.sum(-1, keepdim=True)) + po.sum(-1, keepdim=True)
    o = (over(torch.matmul(pp, vp)) + torch.matmul(po, vo)) / torch.where(total == 0, 1.0, total)
    return o.reshape(b, -1, d).to(DTYPES[c["dtype"]]), (m + torch.log(total)).reshape(b, -1)


def plain_read(s):
    c = s["case"]
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    got = (plain_rows(s[n][page, :, off], None if s[n + "_scales"] is None else s[n + "_scales"][page, :, off], c["cache"])
           for n in ("k", "v"))
    return tuple(x.to(DTYPES[c["dtype"]]) for x in got)


def plain_lora(s):
    """All adapters' products side by side; a token keeps its own adapter's."""
    c = s["case"]
    t, a, r = c["tokens"], c["adapters"], c["rank"]
    h = torch.matmul(s["x"].float(), s["a"].float().view(a * r, -1).t()).view(t, a, r) * s["scales"][None, :, None]
    h = torch.where((s["ids"][:, None] == torch.arange(a, device=DEV))[:, :, None], h, 0.0)
    delta = torch.matmul(h.view(t, a * r), s["b"].float().transpose(1, 2).reshape(a * r, -1))
    return (s["base"].float() + delta).to(DTYPES[c["y"]])


def plain_logprobs(s):
    c = s["case"]
    z = s["logits"].float()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(1)
    entropy = torch.log(total.squeeze(1)) - (e * (z - m).clamp(min=-1e30)).sum(1) / total.squeeze(1)
    got = z.gather(1, s["target"][:, None]).squeeze(1) - lse, lse, entropy
    if not c["top"]:
        return got
    bits = z.contiguous().view(torch.int32)                         # order by value, then by the lower index
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() << 32 | (c["vocab"] - 1 - torch.arange(c["vocab"], device=DEV))
    ids = c["vocab"] - 1 - (torch.topk(key, c["top"], 1).values & 0xffffffff)
    return *got, z.gather(1, ids) - lse[:, None], ids


def plain_logprobs_grad(s):
    z = s["logits"].float()
    lp = z - s["lse"][:, None]
    p = torch.exp(lp)
    dz = -p * (s["d_logprob"][:, None] + s["d_entropy"][:, None] * (lp.clamp(min=-1e30) + s["entropy"][:, None]))
    dz.scatter_add_(1, s["target"][:, None], s["d_logprob"][:, None])
    return dz.to(DTYPES[s["case"]["dtype"]])


def run_plain(s):
    op = s["case"]["op"]
    if op == "shared":
        return plain_shared(s)
    if op == "read":
        return plain_read(s)
    if op == "lora":
        return plain_lora(s)
    return plain_logprobs(s) if op == "logprobs" else plain_logprobs_grad(s)


# ---- the definitions in 64 bits -------------------------------------------------
def value64(codes, bits, man, bias):
    """The value of a sign-magnitude minifloat code."""
    codes = codes.long()
    mag = codes & ((1 << (bits - 1)) - 1)
    e, m = mag >> man, (mag & ((1 << man) - 1)).double() / (1 << man)
    v = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((e - bias).double()))
    return torch.where((codes >> (bits - 1)) & 1 == 1, -v, v)


def rows64(s, name, pages, h, n):
    """The first n tokens of head h on `pages`."""
    x, kind = s[name][pages, h].flatten(0, 1)[:n], s["case"]["cache"]
    if kind == "bf16":
        return x.double()
    if kind == "mxfp4":
        wide = x.new_empty(n, 2 * x.shape[1])
        wide[:, 0::2], wide[:, 1::2] = x % 16, x // 16
        v = value64(wide, 4, 1, 1)
    else:
        v = value64(x, 8, 3, 7)
    e = s[name + "_scales"][pages, h].flatten(0, 1)[:n].int() - 127
    return v * torch.ldexp(torch.ones_like(e, dtype=torch.float64), e).repeat_interleave(32, 1)


def exact_shared(s):
    c = s["case"]
    group = c["hq"] // c["hk"]
    o = torch.zeros(c["batch"], c["hq"], c["dim"], device=DEV, dtype=torch.float64)
    lse = torch.full((c["batch"], c["hq"]), -math.inf, device=DEV, dtype=torch.float64)
    for h in range(c["hk"]):
        kp, vp = (rows64(s, x, s["prefix"].long(), h, c["prefix"]) for x in ("k", "v"))
        for b, n in enumerate(lengths_of(c)):
            pages = s["table"][b, : -(-n // c["page"])].long()
            heads = slice(h * group, (h + 1) * group)
            q = s["q"][b, heads].double()
            z = torch.mm(q, kp.t().contiguous())
            if n:
                z = torch.cat((z, torch.mm(q, rows64(s, "k", pages, h, n).t().contiguous())), 1)
            z = z * s["scale"]
            p = torch.softmax(z, 1)
            lse[b, heads] = torch.logsumexp(z, 1)
            o[b, heads] = torch.mm(p[:, : c["prefix"]].contiguous(), vp)
            if n:
                o[b, heads] += torch.mm(p[:, c["prefix"]:].contiguous(), rows64(s, "v", pages, h, n))
    return o, lse


def exact_read(s):
    """The pages in order, each whole, then cut to the tokens."""
    c = s["case"]
    pages = s["slots"][:: c["page"]] // c["page"]
    return tuple(torch.stack([rows64(s, n, pages, h, c["tokens"]) for h in range(c["hk"])], 1) for n in ("k", "v"))


def exact_lora(s):
    y = s["base"].double()
    for a in range(s["case"]["adapters"]):
        at = torch.nonzero(s["ids"] == a).squeeze(1)
        h = torch.mm(s["x"][at].double(), s["a"][a].double().t().contiguous())
        y[at] += torch.mm(h, s["b"][a].double().t().contiguous()) * s["scales"][a].double()
    return y


def exact_logprobs(s):
    c = s["case"]
    z = s["logits"].double()
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    entropy = -torch.special.xlogy(p := torch.exp(lp), p).sum(1)
    got = lp.gather(1, s["target"][:, None]).squeeze(1), lse, entropy
    if not c["top"]:
        return got
    values, ids = torch.sort(lp, dim=1, descending=True, stable=True)
    return *got, values[:, : c["top"]].contiguous(), ids[:, : c["top"]].contiguous()


def exact_logprobs_grad(s):
    """Through the derivative of p ln p: d(-sum p ln p)/dz = -p (ln p + entropy)."""
    out = torch.empty(s["logits"].shape, device=DEV, dtype=torch.float64)
    for i in range(0, out.shape[0], 512):
        rows = slice(i, i + 512)
        p = torch.exp(s["logits"][rows].double() - s["lse"][rows, None].double())
        chosen = torch.zeros_like(p)
        chosen[torch.arange(p.shape[0], device=DEV), s["target"][rows]] = 1
        out[rows] = s["d_logprob"][rows, None].double() * (chosen - p) - \
            s["d_entropy"][rows, None].double() * (torch.special.xlogy(p, p) + p * s["entropy"][rows, None].double())
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "shared":
        return exact_shared(s)
    if c["op"] == "read":
        return exact_read(s)
    if c["op"] == "lora":
        return exact_lora(s)
    return exact_logprobs(s) if c["op"] == "logprobs" else exact_logprobs_grad(s)
