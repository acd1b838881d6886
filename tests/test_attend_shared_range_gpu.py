"""Attention behind a shared prefix where a range of the prefix is many tiles
long, and where scores or values lie far from one.

Every definition is in float64 over the cache's dequantized values, decoded here.
Tolerances as derived in test_attend_gpu: u = 2^-23, a score is off by at most
dz = (D + 16) u |scale| sum |q k|, n probabilities of 16 bits (fp32 queries: 24)
are summed in fp32."""
import math

import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_attend_gpu import FORMATS, U
from test_attend_shared_gpu import call

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def decoded(codes, scales, kind):
    """Rows of cached values in float64."""
    if kind == "bf16":
        return codes.double()
    if kind == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).double()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda", dtype=torch.float64)
        v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.double() - 127)[..., None]).flatten(-2)


class Batch:
    """A prefix of kv.shape[0] tokens and own tokens (batch x longest, `lengths`
    of them in use) on scattered pages; kv and own: keys, then values, as heads."""

    def __init__(self, kind, kv, own, lengths, page):
        n, hk, dim = kv.shape[0], kv.shape[1] // 2, kv.shape[2]
        ahead, cols = -(-n // page), -(-max(own.shape[1], 1) // page)
        g = torch.Generator(device="cuda").manual_seed(n)
        order = torch.randperm(ahead + own.shape[0] * cols, generator=g, device="cuda").to(torch.int32)
        self.kind, self.page, self.hk = kind, page, hk
        self.ahead, self.table = order[:ahead].contiguous(), order[ahead:].view(own.shape[0], cols)
        self.pn = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.cache = mx.alloc_kv_cache(FORMATS[kind], ahead + own.shape[0] * cols, page, hk, dim)
        t = torch.arange(n, device="cuda")
        self.slots = self.ahead[t // page].long() * page + t % page
        t = torch.arange(own.shape[1], device="cuda")
        self.own_slots = self.table.long()[:, t // page] * page + t % page
        mx.mx_cache_write(self.cache, kv[:, :hk], kv[:, hk:], self.slots)
        if own.shape[1]:
            flat = own.flatten(0, 1)
            mx.mx_cache_write(self.cache, flat[:, :hk], flat[:, hk:], self.own_slots.reshape(-1))

    def rows(self, name, slots):
        """tokens x heads x dim in float64 at those slots."""
        x, s = getattr(self.cache, name), getattr(self.cache, name + "_scales")
        take = lambda t: None if t is None else t[slots // self.page, :, slots % self.page]
        return decoded(take(x), take(s), self.kind)

    def run(self, q, scale):
        return call(self.cache, self.ahead, self.pn, self.table, self.lengths, q, scale)

    def check(self, q, scale, out, lse):
        b, hq, dim = q.shape
        hk, per = self.hk, hq // self.hk
        k, v = (self.rows(x, self.slots).transpose(0, 1).contiguous() for x in ("k", "v"))                 # heads x tokens x dim
        qh = q.double().view(b, hk, per, dim).transpose(0, 1).reshape(hk, b * per, dim).contiguous()
        z = scale * torch.bmm(qh, k.transpose(1, 2).contiguous())
        dz = (dim + 16) * U * abs(scale) * torch.bmm(qh.abs(), k.abs().transpose(1, 2).contiguous()).amax(2)
        zm = z.abs().amax(2)
        m = z.amax(2)
        width = self.own_slots.shape[1]
        if width:
            ok, ov = (self.rows(x, self.own_slots.reshape(-1)).view(b, width, hk, dim).permute(2, 0, 1, 3).contiguous() for x in ("k", "v"))
            q4 = qh.view(hk * b, per, dim)
            flat = lambda t: t.reshape(hk * b, width, dim)
            zo = (scale * torch.bmm(q4, flat(ok).transpose(1, 2).contiguous())).view(hk, b, per, width)
            dead = (torch.arange(width, device="cuda") >= self.lengths[:, None])[None, :, None]
            dzo = (dim + 16) * U * abs(scale) * torch.bmm(q4.abs(), flat(ok).abs().transpose(1, 2).contiguous()).view(hk, b, per, width)
            dz = torch.maximum(dz, dzo.masked_fill(dead, 0).amax(3).view(hk, -1))
            zm = torch.maximum(zm, zo.abs().masked_fill(dead, 0).amax(3).view(hk, -1))
            zo = zo.masked_fill(dead, -math.inf)
            m = torch.maximum(m, zo.amax(3).view(hk, -1))
            po = torch.exp(zo - m.view(hk, b, per)[..., None]).view(hk * b, per, width)
        p = torch.exp(z - m[..., None])
        total, sums, size = p.sum(2), torch.bmm(p, v), torch.bmm(p, v.abs())
        if width:
            total = total + po.sum(2).view(hk, -1)
            sums = sums + torch.bmm(po, flat(ov)).view(hk, -1, dim)
            size = size + torch.bmm(po, flat(ov).abs()).view(hk, -1, dim)
        want, size = sums / total[..., None], size / total[..., None]
        n = k.shape[1] + width
        parts = 2.0 ** -16 if q.dtype == BF16 else U
        tol = (4 * dz + 16 * U * (1 + zm) + parts + 2 * (n + 64) * U)[..., None] * size
        tol = tol + n * 2.0 ** -122 * v.abs().max()                # tokens that count as 0
        if q.dtype == BF16:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        back = lambda t: t.view(hk, b, per, -1).transpose(0, 1).reshape(b, hq, -1)
        err = ((out.double() - back(want)).abs() / back(tol)).nan_to_num(math.inf).max().item()
        assert err <= 1, f"{err:.2f} of the tolerance"
        w = m + torch.log(total)
        room = back(dz + (n + 64) * U + 16 * U * (1 + zm + w.abs())).squeeze(-1)
        err = ((lse.double() - back(w).squeeze(-1)).abs() / room).nan_to_num(math.inf).max().item()
        assert err <= 1, f"lse: {err:.2f} of the tolerance"


# (key-value heads, batch, group, prefix): a prefix in one tile, a range of
# several, tiles of 64, 128 and 256 rows
FORMS = [(2, 3, 2, 200), (64, 8, 2, 2651), (64, 25, 4, 2651), (64, 70, 4, 1400)]


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("hk,batch,group,prefix", FORMS)
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (96, F32), (256, BF16)])
def test_huge_scores(kind, hk, batch, group, prefix, dim, dtype):
    """Scores of 10^4 to 10^31: the likeliest token's value comes out as it is,
    whatever the rounding of a score is worth, beside rows of ordinary scores.

    Its probability p need not be 1 (below 2^20 a score's rounding is up to 2^-4),
    so fp32 outputs p v / p round: three products of p's exact parts and their
    sums (3 u), two joins' factors, each an exponential and a product, of p v and
    of p (at most 2 u each, 8 u in all), the division: less than 16 u.  The bf16
    value nearest to that is v."""
    print(kind, hk, batch, group, prefix, dim, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(prefix + dim)
    kv = torch.randn(prefix, 2 * hk, dim, generator=g, device="cuda")
    own = torch.randn(batch, 1, 2 * hk, dim, generator=g, device="cuda")
    kv[:, :hk] = 0
    own[:, :, :hk] = 0
    kv[:, :hk, 0] = torch.randint(-6, 7, (prefix, hk), generator=g, device="cuda").float()
    kv[:, :hk, 1] = torch.randn(prefix, hk, generator=g, device="cuda")
    heads = torch.arange(hk, device="cuda")
    top, low = (torch.randint(0, prefix // 2, (hk,), generator=g, device="cuda") + o for o in (0, prefix // 2))
    kv[top, heads], kv[low, heads] = 0, 0
    kv[top, heads, 0], kv[low, heads, 0] = 8.0, -8.0
    kv[:, hk:, :] = torch.where(kv[:, hk:].abs() < 0.01, 0.5, kv[:, hk:])
    made = Batch(kind, kv.to(BF16), own.to(BF16), [1] * batch, 16)
    k, v = made.rows("k", made.slots), made.rows("v", made.slots)
    head_of = torch.arange(hk * group, device="cuda") // group
    for e in (16, 21, 25, 30, 31, 33, 40, 100):
        q = torch.zeros(batch, hk * group, dim, device="cuda")
        q[:, :, 1] = torch.randn(batch, hk * group, generator=g, device="cuda")
        usual = torch.rand(batch, hk * group, generator=g, device="cuda") < 0.3
        sign = torch.where(torch.rand(batch, hk * group, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        q[:, :, 0] = torch.where(usual, 0.0, sign * 1.375 * 2.0 ** e)
        q[:, :, 1] *= usual
        q = q.to(dtype)
        for scale in (0.3, -0.7):
            out, lse = made.run(q, scale)
            z = scale * q.double()[..., 0] * torch.where(sign * scale > 0, 8.0, -8.0)
            at = torch.where(sign * scale > 0, top[head_of], low[head_of])
            want = v[at, head_of.expand(batch, -1)].to(dtype)
            near = (out.double() - want.double()).abs() <= (0 if dtype == BF16 else 16 * U) * want.double().abs()
            bad = (~(near | usual[..., None])).any(-1).sum().item()
            assert bad == 0, f"2^{e} x {scale}: {bad} rows"
            # a product with the scale, one with log2 e, one back
            off = ((lse.double() - z).abs() / z.abs().clamp(min=1e-30))[~usual].max().item()
            assert off <= 4 * U, f"2^{e} x {scale}: lse off by {off / U:.1f} u"
            zu = scale * q.double()[..., 1][..., None] * k[:, head_of, 1].t()[None]
            zu = torch.cat((zu, torch.zeros_like(zu[..., :1])), -1)                # the own token's key is zero
            room = (prefix + 64 + dim + 100) * U * (1 + zu.abs().amax(-1))
            off = ((lse.double() - torch.logsumexp(zu, -1)).abs() / room)[usual].max().item()
            assert off <= 1, f"2^{e} x {scale}: the others' lse at {off:.1f} of the tolerance"


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("hk,batch,group,prefix", FORMS[1:])
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (128, F32), (256, BF16)])
def test_values_near_the_largest(kind, hk, batch, group, prefix, dim, dtype):
    """A later token 2^1 to 2^12 times as likely as those before it, with a value
    near fp32's largest: the weighted sum is finite, and comes out so."""
    print(kind, hk, batch, group, prefix, dim, dtype, flush=True)
    kv = torch.zeros(prefix, 2 * hk, dim, device="cuda", dtype=BF16)
    g = torch.Generator(device="cuda").manual_seed(prefix)
    heads = torch.arange(hk, device="cuda")
    late = torch.randint(0, prefix, (hk,), generator=g, device="cuda")
    kv[late, heads, 0] = 1.0
    kv[late, hk + heads] = 1.5 * 2.0 ** 126
    made = Batch(kind, kv, kv.new_zeros(batch, 0, 2 * hk, dim), [0] * batch, 16)
    q = torch.zeros(batch, hk * group, dim, device="cuda", dtype=dtype)
    q[:, :, 0] = torch.arange(batch * hk * group, device="cuda").view(batch, -1) % 12 + 1
    out, lse = made.run(q, math.log(2.0))
    made.check(q, math.log(2.0), out, lse)


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, F32)])
def test_values_near_the_smallest(kind, dim, dtype):
    """Equal values of 1.5 x 2^-120: what a probability below 2^-6 leaves of one
    is subnormal and counts."""
    hk, batch, group, prefix = FORMS[2]
    g = torch.Generator(device="cuda").manual_seed(prefix)
    kv = torch.randn(prefix, 2 * hk, dim, generator=g, device="cuda").to(BF16)
    kv[:, hk:] = 1.5 * 2.0 ** -120
    made = Batch(kind, kv, kv.new_zeros(batch, 0, 2 * hk, dim), [0] * batch, 16)
    q = torch.randn(batch, hk * group, dim, generator=g, device="cuda").to(dtype)
    out, lse = made.run(q, dim ** -0.5)
    made.check(q, dim ** -0.5, out, lse)


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("hk,batch,group,prefix", FORMS)
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, F32), (256, BF16)])
def test_tokens_hardly_likely(kind, hk, batch, group, prefix, dim, dtype):
    """The likeliest token's value is 0: what a token 2^-60 to 2^-121 times as
    likely adds is the whole output, wherever the two lie.

    One probability of 16 or 24 bits times an exact value, two joins' factors and
    a division: 16 u, for bf16 2^-16 and half a unit more."""
    print(kind, hk, batch, group, prefix, dim, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(prefix)
    kv = torch.zeros(prefix, 2 * hk, dim, device="cuda", dtype=BF16)
    heads = torch.arange(hk, device="cuda")
    first = torch.randint(0, prefix // 2, (hk,), generator=g, device="cuda")
    second = torch.randint(prefix // 2, prefix, (hk,), generator=g, device="cuda")
    swap = torch.rand(hk, generator=g, device="cuda") < 0.5
    top, other = torch.where(swap, first, second), torch.where(swap, second, first)
    kv[:, :hk, 0] = -4.0                                  # everyone else: 2^-500 or less
    kv[top, heads, 0], kv[other, heads, 0] = 1.0, 0.0
    kv[other, hk + heads] = 1.0
    made = Batch(kind, kv, kv.new_zeros(batch, 0, 2 * hk, dim), [0] * batch, 16)
    q = torch.zeros(batch, hk * group, dim, device="cuda")
    q[:, :, 0] = torch.tensor([60.0, 100.0, 110.0, 118.0, 121.0], device="cuda")[torch.arange(batch * hk * group, device="cuda") % 5].view(batch, -1)
    # log2 e times fp32's ln 2 is off by u, 121 u in the exponent
    scale = math.log(2.0)
    out, lse = made.run(q.to(dtype), scale)
    want = torch.exp2(-q[:, :, :1].double())
    tol = 16 * U + 2 * U * 121 * math.log(2.0) + (2.0 ** -16 + 2.0 ** -8 if dtype == BF16 else 0)
    off = ((out.double() - want).abs() / want).max().item()
    assert off <= tol, f"off by {off / tol:.2f} of the tolerance"


# (key-value heads, batch, group): 64, 128 and 256 rows to a tile where the
# operands allow it, two tiles of rows in the last; ranges of 650 tokens or more
LONG = [(64, 8, 2), (64, 25, 4), (64, 70, 4)]


def long_batch(kind, hk, batch, group, dim, dtype, page, prefix=2651, seed=0):
    """Scores that climb, fall or jump along the prefix by up to 2^6 each 97
    tokens, head by head, and heads of scores alike."""
    g = torch.Generator(device="cuda").manual_seed(seed + dim + batch)
    kv = torch.randn(prefix, 2 * hk, dim, generator=g, device="cuda")
    step = torch.arange(prefix, device="cuda") // 97
    jumps = torch.randperm(int(step[-1]) + 1, generator=g, device="cuda")
    courses = torch.stack((step, step[-1] - step, jumps[step], 0 * step)).float() * 3
    kv[:, :hk, 0] = courses[torch.arange(hk, device="cuda") % 4].t()
    own = torch.randn(batch, 20, 2 * hk, dim, generator=g, device="cuda")
    lengths = torch.randint(0, 21, (batch,), generator=g, device="cuda").tolist()
    q = torch.randn(batch, hk * group, dim, generator=g, device="cuda")
    q[:, :, 0] = 2 + 4 * torch.rand(batch, hk * group, generator=g, device="cuda")
    return Batch(kind, kv.to(BF16), own.to(BF16), lengths, page), q.to(dtype)


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("hk,batch,group", LONG)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_long_ranges(kind, hk, batch, group, dtype, dim):
    """Ranges of five to dozens of tiles, odd and even counts, a ragged end: the
    maximum moves often, what was summed before is scaled down and counts."""
    print(kind, hk, batch, group, dtype, dim, flush=True)
    made, q = long_batch(kind, hk, batch, group, dim, dtype, 16)
    out, lse = made.run(q, 0.25)
    made.check(q, 0.25, out, lse)


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("hk,batch,group", LONG)
@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, F32), (256, BF16)])
@pytest.mark.parametrize("page", [1, 3])
def test_more_pages_than_are_held(kind, hk, batch, group, dim, dtype, page):
    """Ranges of more pages than a workgroup holds at a time, refilled between tiles."""
    print(kind, hk, batch, group, dim, dtype, page, flush=True)
    made, q = long_batch(kind, hk, batch, group, dim, dtype, page, prefix=4500 * page + 7)
    out, lse = made.run(q, 0.25)
    made.check(q, 0.25, out, lse)
