"""The decode-step operators together, as examples/decode_step.py uses them:
against float64, in a replayed HIP graph, and on a side stream.

Tolerance against float64.  The layer rounds to bf16 (2^-9 of a value) the
projected heads, the rotated ones, the attention's output and its own; the
cache's values are read back as they are.  A relative error e of queries and
keys moves a score by at most 2 e |z|, a probability by a factor of 1 + 4 e |z|
(its own and the sum's).  With |z| below 8 (checked) and e = 2 * 2^-9, that is
1/16 at the very most for one weight, and independent over hundreds of weights
and heads: 3% of the output's norm is well above what rounding gives and far
below any misplaced head, token or scale."""
import os
import sys

import numpy as np
import pytest
import torch

import microscaling_block_quantization_amd as mx

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def dequantized(fmt, q):
    return mx.mx_dequantize(fmt, q).double().cpu().numpy()


def cached(layer, which):
    """pages x heads x page x dim of the cache in float64"""
    c = layer.cache
    t = c.k if which == "k" else c.v
    if c.fmt is None:
        return t.double().cpu().numpy()
    rows = c.pages * c.heads * c.page_size
    q = mx.QTensor(rows, c.dim, t, c.k_scales if which == "k" else c.v_scales)
    return dequantized(c.fmt, q).reshape(c.pages, c.heads, c.page_size, c.dim)


def step64(layer, x, positions, table, lengths):
    """The layer in float64 over what its cache holds."""
    h, hk, d = layer.heads, layer.kv_heads, layer.dim
    x = x.double().cpu().numpy()
    q = (x @ dequantized(layer.fmt, layer.w_qkv).T).reshape(len(x), h + 2 * hk, d)[:, :h]
    q = q / np.sqrt((q * q).mean(-1, keepdims=True) + 1e-6) * layer.q_norm.double().cpu().numpy()
    p = positions.cpu().numpy()
    cos, sin = (t.double().cpu().numpy()[p][:, None] for t in (layer.cos, layer.sin))
    a, b = q[..., :d // 2], q[..., d // 2:]
    q = np.concatenate((a * cos - b * sin, b * cos + a * sin), -1)
    K, V = cached(layer, "k"), cached(layer, "v")
    page, tab = layer.cache.page_size, table.cpu().numpy()
    out = np.zeros((len(x), h, d))
    zmax = 0.0
    for i, n in enumerate(lengths.cpu().numpy()):
        if n == 0:
            continue
        t = np.arange(n)
        for j in range(h):
            k, v = K[tab[i, t // page], j * hk // h, t % page], V[tab[i, t // page], j * hk // h, t % page]
            z = k @ q[i, j] * d ** -0.5
            zmax = max(zmax, np.abs(z).max())
            w = np.exp(z - z.max())
            out[i, j] = w @ v / w.sum()
    return out.reshape(len(x), h * d) @ dequantized(layer.fmt, layer.w_out).T, zmax


def tokens(layer, batch, steps, seed, empty=None):
    """Inputs of `steps` steps; sequence `empty` never gets a token (its slot is
    outside the cache and its length 0)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    page = layer.cache.page_size
    per = -(-steps // page)
    table = torch.randperm(layer.cache.pages, generator=g, device="cuda")[:batch * per].view(batch, per).to(torch.int32)
    for t in range(steps):
        x = torch.randn(batch, 512, generator=g, device="cuda").to(torch.bfloat16)
        at = torch.full((batch,), t, device="cuda", dtype=torch.int32)
        slots = table[:, t // page].long() * page + t % page
        lengths = at + 1
        if empty is not None:
            slots[empty], lengths[empty] = -1, 0
        yield x, at, slots, table, lengths


@pytest.mark.parametrize("fmt,cache_fmt", [(mx.MXFP4, None), (mx.MXFP4, mx.MXFP8_E4M3),
                                           (mx.Format(scale=mx.SCALE_NVFP4, block_cols=16), mx.MXFP4),
                                           (mx.Format(elem=mx.ELEM_INT4, asymmetric=1, rule=mx.RULE_CEIL, block_cols=128), None)],
                         ids=["mxfp4-bf16", "mxfp4-mxfp8", "nvfp4-mxfp4", "int4-bf16"])
def test_layer(fmt, cache_fmt):
    from decode_step import AttentionLayer
    layer = AttentionLayer(512, 8, 2, 128, fmt=fmt, cache_fmt=cache_fmt, pages=40, page_size=16, seed=1)
    for i, args in enumerate(tokens(layer, 5, 70, seed=2, empty=3)):
        y = layer.step(*args)
        if i in (0, 1, 17, 69):
            x, at, _, table, lengths = args
            want, zmax = step64(layer, x, at, table, lengths)
            assert zmax < 8
            got = y.double().cpu().numpy()
            assert (got[3] == 0).all()
            err = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert err < 0.03, f"step {i}: {err:.4f}"


def test_graph_replays():
    """A captured step, its inputs renewed between replays, with eager steps of
    another layer and synchronizations between: every replay's output and cache
    are the eager layer's, bit for bit."""
    from decode_step import AttentionLayer
    eager, graphed, other = (AttentionLayer(512, 8, 2, 64, pages=40, page_size=16, seed=s) for s in (3, 3, 4))
    steps = list(tokens(eager, 4, 36, seed=5))
    held = [t.clone() for t in steps[0]]
    for _ in range(2):
        graphed.step(*held)                       # the same token twice: the cache holds it once
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = graphed.step(*held)
    for i, args in enumerate(steps):
        for h, a in zip(held, args):
            h.copy_(a)
        graph.replay()
        other.step(*args)
        if i % 5 == 0:
            torch.cuda.synchronize()
        assert torch.equal(y, eager.step(*args)), f"replay {i}"
    for a, b in ((eager.cache.k, graphed.cache.k), (eager.cache.v_scales, graphed.cache.v_scales)):
        assert torch.equal(a, b)


def test_side_streams():
    """Two layers stepping at once on two streams of their own, their tensors
    made on the main stream."""
    from decode_step import AttentionLayer
    main = torch.cuda.current_stream()
    want, runs = [], []
    for seed in (6, 7):
        a, b = (AttentionLayer(512, 8, 2, 128, pages=40, page_size=16, seed=seed) for _ in range(2))
        steps = list(tokens(a, 3, 20, seed=seed))
        want.append([a.step(*s) for s in steps])
        runs.append((b, steps, torch.cuda.Stream()))
    outs = [[], []]
    for _, _, s in runs:
        s.wait_stream(main)
    for i in range(20):
        for k, (layer, steps, s) in enumerate(runs):
            with torch.cuda.stream(s):
                outs[k].append(layer.step(*steps[i]))
    for _, _, s in runs:
        main.wait_stream(s)
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))


def test_training_gradient_and_example_runs(capsys):
    import decode_step
    decode_step.main()
    assert "tokens for 3 sequences" in capsys.readouterr().out
    dev = torch.device("cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    leaves = [r(9, 4, 64), r(9, 2, 64), 1 + 0.1 * r(64), 1 + 0.1 * r(64)]
    mine = [t.clone().requires_grad_() for t in leaves]
    ref = [t.double().cpu().requires_grad_() for t in leaves]
    cos, sin = decode_step.rotation_tables(32, 64, dev)
    pos = torch.arange(9, device=dev, dtype=torch.int32) * 3
    target = r(9, 6, 64)

    def loss(yq, yk, t):
        return ((torch.cat((yq, yk), 1) - t) ** 2).sum()

    loss(*decode_step.QKRope.apply(mine[0], mine[1], cos, sin, pos, mine[2], mine[3], 1e-6), target).backward()
    c, s = (t.double().cpu()[pos.cpu().long()][:, None] for t in (cos, sin))

    def plain(x, w):
        u = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = u[..., :32], u[..., 32:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    loss(plain(ref[0], ref[2]), plain(ref[1], ref[3]), target.double().cpu()).backward()
    # fp32 throughout: a few hundred roundings of 2^-24 each on sums of like size
    for m, e in zip(mine, ref):
        assert (m.grad.double().cpu() - e.grad).norm() <= 512 * 2.0 ** -24 * e.grad.norm()
