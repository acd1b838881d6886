"""`stream=` on the GPU: the results are the current stream's, bit for bit, and
what a call allocates for its kernels lies in the pool of the stream they run
on."""
import pytest
import torch

import microscaling_block_quantization_amd as mx

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rnd(*s):
    return torch.randn(*s, device="cuda").to(BF16)


class Recorder:
    """The library, with the arguments of its launches kept."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        f = getattr(self.real, name)
        if name.endswith("_size"):
            return f
        return lambda *a: (self.calls.append((name, a)), f(*a))[1]


def pool_of(address):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("an address outside the allocator's segments")


def rope_backward():
    q, k, gq, gk = rnd(9, 4, 128), rnd(9, 2, 128), rnd(9, 4, 128), rnd(9, 2, 128)
    cos, sin = (torch.randn(40, 64, device="cuda") for _ in range(2))
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    qw, kw = rnd(128), rnd(128)
    return lambda **s: mx.mx_qk_rope_backward(gq, gk, q, k, cos, sin, pos, qw, kw, **s), 9


def attend():
    cache = mx.KVCache(None, rnd(80, 2, 16, 64), rnd(80, 2, 16, 64))
    q, n = rnd(2, 4, 64), torch.tensor([600, 17], device="cuda", dtype=torch.int32)
    table = torch.arange(80, device="cuda", dtype=torch.int32).view(2, 40)
    return lambda **s: mx.mx_attend(q, cache, table, n, lse=True, **s), 10


@pytest.mark.parametrize("make", [rope_backward, attend])
def test_workspace_and_outputs(make, monkeypatch):
    call, at = make()
    want = call()
    side = torch.cuda.Stream()
    library = Recorder(mx.lib())
    with monkeypatch.context() as m:
        m.setattr(mx, "lib", lambda: library)
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    (name, args), = library.calls
    assert args[-1] == side.cuda_stream
    assert pool_of(args[at]) == side.cuda_stream, "the workspace is another stream's"
    for a, b in zip(got, want):
        assert torch.equal(a, b)
        assert pool_of(a.data_ptr()) == side.cuda_stream


def test_many_calls_on_a_side_stream():
    """Allocations of the main stream between the calls find none of their memory."""
    call, _ = attend()
    want = call()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(main)
    outs = []
    for _ in range(50):
        outs.append(call(stream=side))
        torch.full((1 << 16,), float("nan"), device="cuda")
    main.wait_stream(side)
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


NVFP4 = mx.Format(scale=mx.SCALE_NVFP4, block_cols=16)


def test_quantize_and_products():
    """The calls around quantization on a side stream: results as on the
    current one, new tensors in the side stream's pool."""
    x, w = rnd(96, 512), rnd(64, 512)

    def all_of(**s):
        q, dq, st = mx.mx_quantize(NVFP4, x, dequant=torch.float32, stats=True, **s)
        (a, b), sts = mx.mx_quantize_many(mx.MXFP4, [x, w], stats=True, **s)
        return [q.codes, q.scales, q.tensor_scale, dq, st, a.codes, b.scales, sts[0], sts[1],
                mx.mx_dequantize(NVFP4, q, **s), mx.mx_gemm(mx.MXFP4, a, mx.MXFP4, b, **s),
                mx.mx_matvec(mx.MXFP4, b, x[:3], **s)]

    want = all_of()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(main)
    got = all_of(stream=side)
    main.wait_stream(side)
    for i, (a, b) in enumerate(zip(got, want)):
        n = 48 if i in (4, 7, 8) else a.numel()                # mx_stats are 48 bytes
        assert torch.equal(a.view(-1)[:n], b.view(-1)[:n]), i
        assert pool_of(a.data_ptr()) == side.cuda_stream, i
    err, db = mx.mx_qsnr(x, x.clone(), stream=side)
    assert err["n"] == x.numel()


def test_inside_a_graph():
    """A captured stream that forks into the given one and joins it again:
    every replay is the eager result, with the main stream's allocations in
    between."""
    call, _ = attend()
    back, _ = rope_backward()
    want = [t.clone() for t in (*call(), *back())]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = (*call(stream=side), *back(stream=side))
        main.wait_stream(side)
    for i in range(5):
        for t in got:
            t.fill_(float("nan"))
        torch.full((1 << 20,), float("nan"), device="cuda")
        graph.replay()
        if i % 2:
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {i}"
