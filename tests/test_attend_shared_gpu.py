"""Attention behind a shared prefix against float64.

The tolerances are the attention's own (see test_attend_gpu): the prefix's and
a sequence's own tokens count as one sequence of n tokens, scores are off by at
most dz = (D + 16) u |scale| sum |q k|, u = 2^-23, probabilities enter the sum as
two bf16 parts (three for fp32 queries), sums of n terms are fp32.  The hardware
exponential gives 0 below 2^-126, which moves a sum by less than n 2^-126 of its
largest term."""
import math

import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_attend_gpu import FORMATS, U, poisoned_cache, values64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def build(kind, prefix, lengths, hk, dim, page, seed=0, extra=1, spread=1.0):
    """A poisoned cache holding a prefix and the sequences' own tokens on
    scattered pages; unused entries of both tables point outside."""
    g = torch.Generator(device="cuda").manual_seed(seed + dim + page)
    every = [prefix] + list(lengths)
    used = [-(-n // page) for n in every]
    pages = sum(used) + 2
    cache = poisoned_cache(kind, pages, page, hk, dim)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    ahead = torch.full((used[0] + extra,), -7, device="cuda", dtype=torch.int32)
    cols = max(used[1:] + [0]) + extra
    table = torch.full((len(lengths), cols + 3), -5, device="cuda", dtype=torch.int32)[:, :cols]
    at = 0
    for i, (n, u) in enumerate(zip(every, used)):
        row = ahead if i == 0 else table[i - 1]
        row[:u] = order[at:at + u]
        at += u
        if n:
            t = torch.arange(n, device="cuda")
            kv = torch.randn(n, 2 * hk, dim, generator=g, device="cuda")
            kv[:, :hk] *= spread
            kv = kv.to(BF16)
            mx.mx_cache_write(cache, kv[:, :hk], kv[:, hk:], (row[t // page].long() * page + t % page).contiguous())
    as_int = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)
    return cache, ahead, as_int([prefix]), table, as_int(list(lengths))


def check(cache, ahead, pn, table, lengths, q, scale, out, lse, label=""):
    k64, v64 = values64(cache, "k"), values64(cache, "v")
    q64, o, ls = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    page = cache.page_size
    clip = lambda n, cols: min(max(int(n), 0), cols * page)
    first = ahead.cpu().numpy()
    tab, n_of = table.cpu().numpy(), lengths.cpu().numpy()
    t = np.arange(clip(pn.item(), len(first)))
    front = first[t // page] * page + t % page if len(t) else t
    batch, hq, dim = q64.shape
    per = hq // cache.heads
    for b in range(batch):
        t = np.arange(clip(n_of[b], tab.shape[1]))
        rows = np.concatenate([front, tab[b, t // page].astype(np.int64) * page + t % page if len(t) else t])
        n = len(rows)
        if n == 0:
            assert (o[b] == 0).all() and (ls[b] == -np.inf).all(), f"{label}: empty row {b}"
            continue
        for kv in range(cache.heads):
            hs = slice(kv * per, (kv + 1) * per)
            K, V = k64[rows // page, kv, rows % page], v64[rows // page, kv, rows % page]
            Q = q64[b, hs]
            z = scale * (Q @ K.T)
            dz = ((dim + 16) * U * abs(scale) * (np.abs(Q) @ np.abs(K).T)).max(1)
            zm = np.abs(z).max(1)
            p = np.exp(z - z.max(1, keepdims=True))
            total = p.sum(1)
            want = p @ V / total[:, None]
            parts = 2.0 ** -16 if out.dtype == BF16 else U
            tol = (4 * dz + 16 * U * (1 + zm) + parts + 2 * (n + 64) * U)[:, None] * (p @ np.abs(V) / total[:, None])
            if out.dtype == BF16:
                tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
            err = np.abs(o[b, hs] - want)
            assert (err <= tol).all(), f"{label} b{b} kv{kv}: {np.max(err / tol):.2f} of the tolerance"
            w = z.max(1) + np.log(total)
            assert (np.abs(ls[b, hs] - w) <= dz + (n + 64) * U + 16 * U * (1 + zm + np.abs(w))).all(), f"{label} b{b} kv{kv}: lse"


def call(cache, ahead, pn, table, n, q, scale=None, **kw):
    ws = mx.alloc_attend_shared_workspace(cache, q.shape[0], q.shape[1], ahead.shape[0], table.shape[1]).fill_(0xFF)
    return mx.mx_attend_shared(q, cache, ahead, pn, table, n, scale=scale, lse=True, workspace=ws, **kw)


def run(kind, prefix, lengths, group, hk, dim, page, dtype, seed=0, scale=None, **kw):
    print(kind, prefix, lengths, group, hk, dim, page, dtype, flush=True)
    made = build(kind, prefix, lengths, hk, dim, page, seed, **kw)
    q = torch.randn(len(lengths), group * hk, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)
    s = dim ** -0.5 if scale is None else scale
    out, lse = call(*made, q, s)
    check(*made, q, s, out, lse, f"{kind} {prefix}+{lengths} {group}x{hk} {dim} page {page}")
    return made, q, out, lse


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_lengths_and_dims(kind, dtype, dim):
    run(kind, 200, [0, 1, 15, 33, 129], 4, 2, dim, 16, dtype)
    run(kind, 1, [40, 0, 7], 1, 3, dim, 24, dtype)


@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1000])
def test_prefix_lengths(prefix):
    run("bf16", prefix, [5, 0, 70], 2, 2, 64, 16, BF16)
    run("mxfp8", prefix, [5, 0, 70], 11, 1, 128, 32, BF16)
    run("mxfp4", prefix, [5, 0, 70], 24, 1, 128, 64, BF16)


@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 128])
def test_page_sizes(kind, page):
    run(kind, 257, [5, 96], 8, 1, 128, page, BF16)


@pytest.mark.parametrize("batch,group", [(1, 1), (31, 1), (8, 4), (3, 11), (32, 2), (13, 5), (16, 8), (43, 3), (150, 2), (9, 33)])
@pytest.mark.parametrize("kind,dtype,dim", [("bf16", BF16, 64), ("mxfp8", F32, 128), ("mxfp4", BF16, 192)])
def test_rows(batch, group, kind, dtype, dim):
    """Every tile of rows, whole and ragged, one and several."""
    rng = np.random.default_rng(batch)
    run(kind, 150, [int(v) for v in rng.integers(0, 40, batch)], group, 2, dim, 16, dtype, seed=batch)


@pytest.mark.parametrize("kind", FORMATS)
def test_long_prefix(kind):
    """A prefix over many workgroups, and one over fewer than there are."""
    run(kind, 9001, [300, 0], 4, 2, 128, 16, BF16)
    run(kind, 5000, [1] * 20, 4, 1, 64, 64, F32)
    run(kind, 4000, [700, 33, 0, 129] * 9, 4, 2, 128, 64, BF16)


def test_peaked_scores():
    """Scores of hundreds: the running maximum grows and old sums vanish."""
    run("bf16", 777, [200, 3], 4, 2, 128, 16, BF16, spread=40.0)
    run("mxfp8", 777, [5, 9], 4, 2, 64, 16, F32, spread=40.0, scale=-0.7)
    run("bf16", 100, [50, 0], 2, 2, 64, 16, BF16, scale=0.0)


def test_no_columns_and_no_sequences():
    made, q, out, lse = run("bf16", 90, [20, 30], 2, 2, 64, 16, BF16)
    cache, ahead, pn, table, n = made
    none = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    got, l2 = call(cache, ahead, pn, none, n, q)
    check(cache, ahead, pn, none, n, q, 64 ** -0.5, got, l2)
    got, l2 = call(cache, ahead[:0], pn, table, n, q)
    check(cache, ahead[:0], pn, table, n, q, 64 ** -0.5, got, l2)
    got, l2 = call(cache, ahead[:0], pn, none, n, q)
    assert (got == 0).all() and (l2 == -math.inf).all()
    assert mx.mx_attend_shared(q[:0], cache, ahead, pn, table[:0], n[:0]).shape == (0, 4, 64)


@pytest.mark.parametrize("page", [16, 10])
def test_lengths_past_the_tables(page):
    """They count as the tables; negative ones as none."""
    (cache, ahead, pn, table, n), q, out, lse = run("bf16", 4 * page, [5, 40, 3 * page], 2, 2, 64, page, BF16, extra=0)
    cache.k.nan_to_num_(0.5)
    cache.v.nan_to_num_(0.5, 0.5, 0.5)
    more = n.clone()
    more[int(n.argmax())] += 1000                         # the one whose pages fill its row of the table
    got, l2 = call(cache, ahead, pn + 1000, table.contiguous(), more, q)
    assert torch.equal(got, out) and torch.equal(l2, lse)
    got, l2 = call(cache, ahead, -pn, table, torch.full_like(n, -3), q)
    assert (got == 0).all() and (l2 == -math.inf).all()


@pytest.mark.parametrize("batch", [3, 40])
def test_bad_pages(batch):
    (cache, ahead, pn, table, n), q, out, lse = run("mxfp8", 300, [20] * batch, 4, 2, 128, 16, BF16)
    bad = table.clone()
    bad[1, 1] = cache.pages
    got, l2 = call(cache, ahead, pn, bad, n, q)
    keep = [b for b in range(batch) if b != 1]
    assert got[1].isnan().all() and l2[1].isnan().all() and torch.equal(got[keep], out[keep])
    for wrong in (-1, cache.pages):
        first = ahead.clone()
        first[18] = wrong
        got, l2 = call(cache, first, pn, table, n, q)
        assert got.isnan().all() and l2.isnan().all()


def test_non_finite_values_in_use():
    """A NaN key of the prefix poisons its head in every sequence, a NaN query its own row."""
    (cache, ahead, pn, table, n), q, out, lse = run("bf16", 100, [5, 60, 0], 2, 2, 128, 16, BF16)
    cache.k[int(ahead[2]), 1, 3, 9] = float("nan")
    got, l2 = call(cache, ahead, pn, table, n, q)
    assert got[:, 2:].isnan().all() and l2[:, 2:].isnan().all() and torch.equal(got[:, :2], out[:, :2])
    cache.k.nan_to_num_(0.25)
    base, _ = call(cache, ahead, pn, table, n, q)
    q2 = q.clone()
    q2[1, 1, 5] = float("inf")
    got, _ = call(cache, ahead, pn, table, n, q2)
    assert got[1, 1].isnan().all()
    keep = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    keep[1, 1] = False
    assert torch.equal(got[keep], base[keep])


def test_against_one_sequence_at_a_time():
    """mx_attend over the prefix's pages and the own ones in one table."""
    (cache, ahead, pn, table, n), q, out, lse = run("mxfp4", 512, [100, 1, 64], 4, 2, 128, 32, BF16, extra=0)
    whole = torch.cat((ahead[None].expand(3, -1), table), 1).contiguous()
    got, l2 = mx.mx_attend(q, cache, whole, n + 512, lse=True)
    assert (got.float() - out.float()).abs().max() <= 2.0 ** -7 * out.float().abs().max()
    assert (l2 - lse).abs().max() < 1e-5


def test_strided_operands_and_same_bits():
    (cache, ahead, pn, table, n), q, out, lse = run("mxfp8", 3000, [300, 20], 4, 2, 128, 16, BF16)
    wide = torch.zeros(2, 3, 8, 128, device="cuda", dtype=BF16)
    wide[:, 1] = q
    dst = torch.full((2, 8, 3, 128), 5.0, device="cuda", dtype=BF16)
    l2 = torch.empty(17, device="cuda")[1:].view(2, 8)
    slice_of = torch.cat((ahead[:1], ahead))[1:]
    for _ in range(3):
        mx.mx_attend_shared(wide[:, 1], cache, slice_of, pn, table, n, out=dst[:, :, 1], lse=l2)
        assert torch.equal(dst[:, :, 1], out) and torch.equal(l2, lse)
    assert (dst[:, :, 0] == 5).all() and (dst[:, :, 2] == 5).all()


def test_workspace_of_a_larger_call():
    """One workspace for every smaller call, and none smaller than asked for."""
    (cache, ahead, pn, table, n), q, out, lse = run("bf16", 400, [30] * 20, 8, 1, 64, 16, BF16)
    big = mx.alloc_attend_shared_workspace(cache, 20, 8, ahead.shape[0], table.shape[1])
    for b in (1, 3, 4, 5, 8, 9, 16, 17, 20):
        for cols in (1, 5, ahead.shape[0]):
            got = mx.mx_attend_shared(q[:b], cache, ahead[:cols], pn, table[:b], n[:b], workspace=big)
            assert torch.equal(got, mx.mx_attend_shared(q[:b], cache, ahead[:cols], pn, table[:b], n[:b]))
    with pytest.raises(mx.MxError):
        mx.mx_attend_shared(q, cache, ahead, pn, table, n, workspace=big[:-16].clone())


def test_graph_with_growing_lengths():
    """A captured step, replayed while lengths, prefix and queries change."""
    (cache, ahead, pn, table, n), q, out, lse = run("bf16", 600, [60, 20, 0, 90], 4, 2, 128, 16, BF16)
    ws = mx.alloc_attend_shared_workspace(cache, 4, 8, ahead.shape[0], table.shape[1])
    at, pl, qs = n.clone(), pn.clone(), q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.mx_attend_shared(qs, cache, ahead, pl, table, at, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, l2 = mx.mx_attend_shared(qs, cache, ahead, pl, table, at, lse=True, workspace=ws)
    for i in range(4):
        at.copy_((n - 7 * i).clamp(min=0))
        pl.fill_(600 - 130 * i)
        qs.copy_(torch.randn_like(q))
        g.replay()
        torch.cuda.synchronize()
        want, wl = mx.mx_attend_shared(qs, cache, ahead, pl, table, at, lse=True)
        assert torch.equal(got, want) and torch.equal(l2, wl)


def test_two_streams_at_once():
    made, q, out, lse = run("mxfp8", 2000, [100] * 12, 4, 2, 128, 16, BF16)
    cache, ahead, pn, table, n = made
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [mx.mx_attend_shared(q, cache, ahead, pn, table, n, lse=True, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_offsets_past_32_bits():
    """A cache over 4 GiB per side, the prefix in its last pages."""
    pages, heads, page, dim = 2200, 4, 2048, 128
    assert pages * heads * page * dim * 2 > 1 << 32
    k = torch.empty((pages, heads, page, dim), dtype=BF16, device="cuda")
    cache = mx.KVCache(None, k, torch.empty_like(k))
    n = 2500
    ahead = torch.tensor([pages - 1, pages - 2], dtype=torch.int32, device="cuda")
    t = torch.arange(n, device="cuda")
    kv = torch.randn(n, 2 * heads, dim, device="cuda").to(BF16)
    slots = ahead[t // page].long() * page + t % page
    mx.mx_cache_write(cache, kv[:, :heads], kv[:, heads:], slots)
    q = torch.randn(3, 8, dim, device="cuda").to(BF16)
    pn, none = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    out, lse = call(cache, ahead, pn, table, none, q)
    small = mx.KVCache(None, k[-2:].clone(), cache.v[-2:].clone())
    check(small, torch.tensor([1, 0]), pn, table, none, q, dim ** -0.5, out, lse, "far pages")
    rk, rv = mx.mx_cache_read(cache, slots)
    assert torch.equal(rk, kv[:, :heads]) and torch.equal(rv, kv[:, heads:])


@pytest.mark.parametrize("kind,heads,batch,group,prefix,same", [("bf16", 8, 75, 4, 40000, True), ("mxfp8", 64, 3, 1, 6000, False),
                                                                ("mxfp4", 32, 20, 4, 12000, True)])
def test_ranges_of_many_pages(kind, heads, batch, group, prefix, same):
    """Pages of one token: a range has more of them than are held at a time.  The
    same tokens on pages of 64 give the same bits where a tile of 32 or 64 tokens
    ends with them, and the same values elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(heads)
    kv = torch.randn(prefix, 2 * heads, 64, generator=g, device="cuda").to(BF16)
    q = torch.randn(batch, heads * group, 64, generator=g, device="cuda").to(BF16)
    got = []
    for page in (1, 64):
        pages = -(-prefix // page)
        cache = mx.alloc_kv_cache(FORMATS[kind], pages, page, heads, 64)
        ahead = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        t = torch.arange(prefix, device="cuda")
        mx.mx_cache_write(cache, kv[:, :heads], kv[:, heads:], ahead[t // page].long() * page + t % page)
        none = torch.zeros(batch, dtype=torch.int32, device="cuda")
        got.append(call(cache, ahead, torch.tensor([prefix], dtype=torch.int32, device="cuda"), none[:, None].contiguous(), none, q))
    (a, la), (b, lb) = got
    if same:
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max() and (la - lb).abs().max() < 1e-5
    # against the definition: the first and the last sequence
    for r in (0, batch - 1):
        for h in (0, heads * group - 1):
            z = torch.mv(kv[:, h // group].double(), q[r, h].double()) * 64 ** -0.5 if kind == "bf16" else None
            if z is not None:
                w = torch.mv(kv[:, heads + h // group].double().t().contiguous(), torch.softmax(z, 0))
                assert (a[r, h].double() - w).abs().max() < 2.0 ** -7 * w.abs().max()
                assert abs(la[r, h].double() - torch.logsumexp(z, 0)) < 1e-4
