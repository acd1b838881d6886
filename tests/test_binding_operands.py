"""What the decode-step calls refuse before anything is launched: operands that
do not lie on the GPU the call runs on, and buffers smaller than what the
kernels read and write.  No GPU: see on_host."""
import pytest
import torch

import microscaling_block_quantization_amd as mx
from on_host import Machine, Stream, gpu

BF16 = torch.bfloat16


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def zeros(*shape, dtype=BF16, card=0):
    return gpu(torch.zeros(*shape, dtype=dtype), card)


def int4():
    return mx.Format(elem=mx.ELEM_INT4, asymmetric=1, rule=mx.RULE_CEIL)


WEIGHTS = {                                      # format, buffers of 32 x 128 weights
    "mxfp4": (mx.Format(), dict(codes=2048, scales=128)),
    "b16": (mx.Format(block_cols=16), dict(codes=2048, scales=256)),
    "nvfp4": (mx.Format(scale=mx.SCALE_NVFP4, block_cols=16), dict(codes=2048, scales=256, tensor_scale=1)),
    "mbs": (mx.Format(macro_cols=128), dict(codes=2048, scales=128, macro_scales=32)),
    "int4 min/max": (int4(), dict(codes=2048, scales=128, offsets=128)),
}
KIND = dict(offsets=torch.int16, tensor_scale=torch.float32)


def weight(kind="mxfp4", card=0, **instead):
    fmt, sizes = WEIGHTS[kind]
    buffers = {n: zeros(s, dtype=KIND.get(n, torch.uint8), card=card) for n, s in sizes.items()}
    return fmt, mx.QTensor(32, 128, **(buffers | instead))


def cache(card=0, pages=80, fmt=None):
    last = {None: 64}.get(fmt, 64)
    if fmt is None:
        return mx.KVCache(None, *(zeros(pages, 2, 16, last, card=card) for _ in range(2)))
    u8 = lambda n: zeros(pages, 2, 16, n, dtype=torch.uint8, card=card)
    return mx.KVCache(fmt, u8(64), u8(64), u8(2), u8(2))


def matvec(card=0, **kw):
    fmt, w = weight(card=card)
    return mx.mx_matvec(fmt, w, kw.pop("x", zeros(3, 128, card=card)), **kw)


def rope_args(card):
    return (zeros(40, 32, dtype=torch.float32, card=card), zeros(40, 32, dtype=torch.float32, card=card),
            zeros(3, dtype=torch.int32, card=card), zeros(64, card=card), zeros(64, card=card))


def rope(card=0, **kw):
    return mx.mx_qk_rope(zeros(3, 4, 64, card=card), zeros(3, 2, 64, card=card), *rope_args(card), **kw)


def rope_backward(card=0, **kw):
    h = lambda n: zeros(3, n, 64, card=card)
    return mx.mx_qk_rope_backward(h(4), h(2), h(4), h(2), *rope_args(card), **kw)


def write(card=0, **kw):
    h = lambda: zeros(3, 2, 64, card=card)
    return mx.mx_cache_write(cache(card), h(), h(), zeros(3, dtype=torch.int64, card=card), **kw)


def attend(card=0, **kw):
    return mx.mx_attend(zeros(2, 4, 64, card=card), cache(card), zeros(2, 30, dtype=torch.int32, card=card),
                        zeros(2, dtype=torch.int32, card=card), **kw)


CALLS = [matvec, rope, rope_backward, write, attend]


@pytest.mark.parametrize("call", CALLS)
def test_on_the_current_gpu(machine, call):
    call()
    assert len(machine.launches) == 1


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors(machine, call):
    with pytest.raises(ValueError, match="GPU"):
        call(card=-1)
    assert not machine.launches


@pytest.mark.parametrize("call", CALLS)
def test_one_operand_on_the_host(machine, call, monkeypatch):
    """Each tensor of the call in turn."""
    made, real = [], globals()["zeros"]
    count = 0

    def nth(*shape, dtype=BF16, card=0):
        made.append(None)
        return real(*shape, dtype=dtype, card=-1 if len(made) == count else card)

    monkeypatch.setitem(globals(), "zeros", nth)
    call()
    for count in range(1, len(made) + 1):
        made.clear()
        machine.launches.clear()
        with pytest.raises(ValueError):
            call()
        assert not machine.launches, f"tensor {count} of the call lay on the host"


@pytest.mark.parametrize("kind", WEIGHTS)
def test_each_buffer_of_a_weight_on_the_host(machine, kind):
    fmt, sizes = WEIGHTS[kind]
    x = zeros(3, 128)
    mx.mx_matvec(fmt, weight(kind)[1], x)
    for name, n in sizes.items():
        _, w = weight(kind, **{name: zeros(n, dtype=KIND.get(name, torch.uint8), card=-1)})
        with pytest.raises(ValueError):
            mx.mx_matvec(fmt, w, x)
    assert len(machine.launches) == 1


@pytest.mark.parametrize("call", [rope_backward, attend])
def test_workspace_on_the_host_or_with_gaps(machine, call):
    call(workspace=zeros(1 << 22, dtype=torch.uint8))
    for bad in (zeros(1 << 22, dtype=torch.uint8, card=-1), zeros(1 << 23, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=bad)
    assert len(machine.launches) == 1


def test_workspace_bytes(machine):
    """A workspace of any type counts by its bytes."""
    attend(workspace=zeros(1 << 20, dtype=torch.float32))
    assert 4 << 20 in machine.launches[0][1]


@pytest.mark.parametrize("kind", WEIGHTS)
def test_weight_buffers_too_small(machine, kind):
    """One byte (or value) less than rows, columns and format need, each buffer in turn."""
    fmt, sizes = WEIGHTS[kind]
    x = zeros(3, 128)
    for name, n in sizes.items():
        dtype = KIND.get(name, torch.uint8)
        mx.mx_matvec(fmt, weight(kind, **{name: zeros(n + 5, dtype=dtype)})[1], x)       # more than enough
        machine.launches.clear()
        with pytest.raises(ValueError, match=name):
            mx.mx_matvec(fmt, weight(kind, **{name: zeros(n - 1, dtype=dtype)})[1], x)
        assert not machine.launches, name


def test_tensor_scale_of_another_type(machine):
    fmt, w = weight("nvfp4", tensor_scale=zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="tensor_scale"):
        mx.mx_matvec(fmt, w, zeros(3, 128))
    assert not machine.launches


@pytest.mark.parametrize("fmt", [mx.MXFP8_E4M3, mx.Format(block_rows=32, block_cols=32), mx.Format(block_cols=0),
                                 mx.Format(block_cols=24), mx.Format(elem=mx.ELEM_INT4, asymmetric=1)])
def test_formats_and_missing_buffers_stay_the_library_s_to_refuse(fmt):
    """The real library: formats without a kernel, and an absent buffer."""
    import ctypes
    u8 = torch.zeros(4096, dtype=torch.uint8)
    f, q = fmt.c(), mx.QTensor(32, 128, u8, u8).c()
    rc = mx.lib().mx_matvec(ctypes.byref(f), ctypes.byref(q), 1, u8.data_ptr(), 1, 128, None, u8.data_ptr(), 32, 1, None)
    assert rc in (mx.MX_ERR_UNSUPPORTED, mx.MX_ERR_ARG)


@pytest.mark.parametrize("fmt", [mx.MXFP8_E4M3, mx.Format(block_rows=32, block_cols=32), mx.Format(block_cols=0)])
def test_formats_without_a_kernel_reach_the_library(machine, fmt):
    w = mx.QTensor(32, 128, zeros(16, dtype=torch.uint8), zeros(1, dtype=torch.uint8))
    mx.mx_matvec(fmt, w, zeros(3, 128))
    assert len(machine.launches) == 1


@pytest.mark.parametrize("call", CALLS)
def test_another_gpu_than_the_current_one(machine, call):
    """Operands of GPU 1 under a launch on GPU 0, by the current device and by
    a stream of GPU 0; and on GPU 1 both ways."""
    with pytest.raises(ValueError, match="device"):
        call(card=1)
    with pytest.raises(ValueError, match="device"):
        call(card=1, stream=Stream(2, device=0))
    with pytest.raises(ValueError, match="device"):
        call(stream=Stream(7, device=1))
    assert not machine.launches
    call(card=1, stream=Stream(7, device=1))
    machine.device = 1
    call(card=1)
    assert len(machine.launches) == 2
