"""`stream=` of the Python calls: what a call allocates for itself belongs to
the stream its kernels run on (it returns to the allocator when the call
returns, while they may still run), and so do its outputs, whose use on the
caller's stream is recorded.  No GPU: see on_host."""
import ctypes

import pytest
import torch

import microscaling_block_quantization_amd as mx
from on_host import Machine, OnGpu, Stream, gpu

BF16 = torch.bfloat16


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def weight(n=64, k=256, fmt=mx.MXFP4):
    return mx.QTensor(n, k, gpu(torch.zeros(n * k // 2, dtype=torch.uint8)),
                      gpu(torch.zeros(n * k // fmt.block_cols, dtype=torch.uint8)))


def heads(t, h, d=64, dtype=BF16):
    return gpu(torch.zeros(t, h, d, dtype=dtype))


def table(rows=40, half=32):
    return gpu(torch.zeros(rows, half))


def cache(pages=80, page=16, h=2, d=64):
    return mx.KVCache(None, *(gpu(torch.zeros(pages, h, page, d, dtype=BF16)) for _ in range(2)))


def ints(n, dtype=torch.int32):
    return gpu(torch.zeros(n, dtype=dtype))


def norm(d=64):
    return gpu(torch.zeros(d, dtype=BF16))


def matvec(stream):
    return mx.mx_matvec(mx.MXFP4, weight(), gpu(torch.zeros(3, 256, dtype=BF16)), stream=stream)


def rope(stream):
    return mx.mx_qk_rope(heads(3, 4), heads(3, 2), table(), table(), ints(3), norm(), norm(), stream=stream)


def rope_backward(stream):
    return mx.mx_qk_rope_backward(heads(3, 4), heads(3, 2), heads(3, 4), heads(3, 2), table(), table(), ints(3), norm(), norm(),
                                  stream=stream)


def attend(stream):
    return mx.mx_attend(heads(2, 4), cache(), gpu(torch.zeros(2, 30, dtype=torch.int32)), ints(2), lse=True, stream=stream)


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    if isinstance(out, mx.QTensor):
        return tensors([out.codes, out.scales, out.offsets, out.macro_scales, out.tensor_scale, out.ref_exp])
    return [t for o in out if o is not None for t in tensors(o)] if isinstance(out, (list, tuple)) else []


def addresses(args):
    """The tensors' addresses among a call's arguments, structs looked into."""
    for a in args:
        if isinstance(a, ctypes.c_void_p):
            yield a.value
        elif isinstance(a, int):
            yield a
        elif isinstance(a, bytes):
            yield from memoryview(a[:len(a) // 8 * 8]).cast("Q")
        elif isinstance(a, ctypes.Array) and issubclass(a._type_, ctypes.Structure):
            for e in a:
                yield from (v for v in (getattr(e, n) for n, _ in e._fields_) if isinstance(v, int))


def number(stream):
    return stream.value if isinstance(stream, ctypes.c_void_p) else stream


def check(machine, call):
    side = Stream(2)
    out = call(side)
    (name, args), = machine.launches
    assert number(args[-1]) == 2, "launched on another stream"
    used = {a for a in addresses(args) if a in machine.allocated}
    assert used, "the call allocated nothing, so the test shows nothing"
    for a in used:
        assert machine.allocated[a][0] == 2, f"{name}: memory of the caller's stream under a launch on another"
    for t in tensors(out):
        assert 1 in getattr(t, "recorded", ()), f"{name}: an output the caller's stream may use is not recorded there"
    assert machine.stream.cuda_stream == 1


@pytest.mark.parametrize("call", [matvec, rope, rope_backward, attend])
def test_decode_calls(machine, call):
    check(machine, call)


@pytest.mark.parametrize("call", [matvec, rope, rope_backward, attend])
def test_the_current_stream_given_by_name(machine, call):
    """Same stream, nothing to record."""
    out = call(Stream(1))
    assert number(machine.launches[0][1][-1]) == 1
    assert all(not getattr(t, "recorded", ()) for t in tensors(out))


# ---- quantization, its inverse, statistics, the large product -------------------
STATS = mx.Format(scale=mx.SCALE_NVFP4, block_cols=16)


def quantize(stream):
    return mx.mx_quantize(STATS, heads(1, 64, 128)[0], dequant=torch.float32, stats=True, stream=stream)


def quantize_many(stream):
    outs, stats = mx.mx_quantize_many(STATS, [heads(1, 64, 128)[0], heads(1, 32, 64)[0]], stats=True, stream=stream)
    return outs + stats


def dequantize(stream):
    return mx.mx_dequantize(mx.MXFP4, weight(), stream=stream)


def gemm(stream):
    return mx.mx_gemm(mx.MXFP4, weight(32), mx.MXFP4, weight(64), stream=stream)


def qsnr(stream):
    return mx.mx_qsnr(heads(1, 64, 128)[0], heads(1, 64, 128)[0], stream=stream)


@pytest.mark.parametrize("call", [quantize, quantize_many, dequantize, gemm, qsnr])
def test_other_calls(machine, call):
    check(machine, call)


def test_quantize_noalloc_allocates_nothing(machine):
    q = mx.alloc_qtensor(mx.MXFP4, 64, 256)
    made = len(machine.allocated)
    out, _, _ = mx.mx_quantize_noalloc(mx.MXFP4, heads(1, 64, 256)[0], q, stream=Stream(2))
    assert out is q and len(machine.allocated) == made and number(machine.launches[0][1][-1]) == 2
