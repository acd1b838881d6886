"""The decode step in replayed HIP graphs and on two streams at sizes where a
sequence is shared out over workgroups (a workspace, a second launch that joins
it) and the products take the long-K kernel."""
import pytest
import torch

import microscaling_block_quantization_amd as mx
from test_decode_step_gpu import dequantized, step64  # also puts the examples on the path

pytestmark = pytest.mark.gpu
HIDDEN = 4096                                  # from 4096 on bf16 products split K over spans
PAGE, COLUMNS = 16, 40                         # tables of 640 tokens


def layer_of(seed, cache_fmt=mx.MXFP8_E4M3):
    from decode_step import AttentionLayer
    a = AttentionLayer(HIDDEN, 8, 2, 128, cache_fmt=cache_fmt, pages=3 * COLUMNS, page_size=PAGE, max_batch=3,
                       table_cols=COLUMNS, seed=seed)
    assert a.workspace.numel() > 0
    return a


def filled(layer, seed):
    """Sequences of 600, 130 and 0 tokens already in the cache."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randperm(3 * COLUMNS, generator=g, device="cuda").view(3, COLUMNS).to(torch.int32)
    start = [600, 130, 0]
    for b, n in enumerate(start):
        if n:
            t = torch.arange(n, device="cuda")
            kv = torch.randn(n, 4, 128, generator=g, device="cuda").to(torch.bfloat16)
            mx.mx_cache_write(layer.cache, kv[:, :2], kv[:, 2:], table[b, t // PAGE].long() * PAGE + t % PAGE)
    return table, torch.tensor(start, device="cuda", dtype=torch.int32)


def steps_of(table, start, count, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.arange(3, device="cuda")
    for i in range(count):
        at = start + i
        x = torch.randn(3, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        slots = table[rows, (at // PAGE).long()].long() * PAGE + at % PAGE
        yield x, at, slots, table, at + 1


def test_against_float64():
    layer = layer_of(1)
    table, start = filled(layer, 2)
    for i, args in enumerate(steps_of(table, start, 3, 3)):
        y = layer.step(*args)
        want, zmax = step64(layer, args[0], args[1], table, args[4])
        assert zmax < 8
        got = y.double().cpu().numpy()
        assert ((got - want) ** 2).sum() ** 0.5 < 0.03 * (want ** 2).sum() ** 0.5, f"step {i}"


def test_graph_replays():
    """Every replay is the eager step's, bit for bit, with the workspace filled
    with NaN before it and eager steps of another layer in between."""
    eager, graphed, other = layer_of(4), layer_of(4), layer_of(5)
    (table, start), _, _ = filled(eager, 6), filled(graphed, 6), filled(other, 6)
    steps = list(steps_of(table, start, 12, 7))
    held = [t.clone() for t in steps[0]]
    for _ in range(2):
        graphed.step(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = graphed.step(*held)
    for i, args in enumerate(steps):
        for h, a in zip(held, args):
            h.copy_(a)
        graphed.workspace.fill_(0xFF)
        graph.replay()
        other.step(*args)
        if i % 5 == 0:
            torch.cuda.synchronize()
        assert torch.equal(y, eager.step(*args)), f"replay {i}"
    assert torch.equal(eager.cache.k, graphed.cache.k) and torch.equal(eager.cache.v_scales, graphed.cache.v_scales)


def test_two_streams():
    """Two layers, each with its workspace, at once on two streams."""
    main = torch.cuda.current_stream()
    want, runs = [], []
    for seed, fmt in ((8, None), (9, mx.MXFP4)):
        a, b = layer_of(seed, fmt), layer_of(seed, fmt)
        (table, start), _ = filled(a, seed), filled(b, seed)
        steps = list(steps_of(table, start, 10, seed))
        want.append([a.step(*s) for s in steps])
        b.workspace.fill_(0xFF)
        runs.append((b, steps, torch.cuda.Stream()))
    outs = [[], []]
    for _, _, s in runs:
        s.wait_stream(main)
    for i in range(10):
        for k, (layer, steps, s) in enumerate(runs):
            with torch.cuda.stream(s):
                outs[k].append(layer.step(*steps[i]))
    for _, _, s in runs:
        main.wait_stream(s)
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))
