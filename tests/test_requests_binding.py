"""The Python calls that serve many requests, without a GPU (see on_host):
operands off the GPU or on another one, shapes and buffers that do not fit,
allocations by stream, autograd's count of changes."""
import pytest
import torch

import microscaling_block_quantization_amd as mx
import on_host
from on_host import Machine, Stream, gpu
from test_binding_streams import cache, check, heads, ints, number

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def machine(monkeypatch):
    monkeypatch.setattr(on_host, "SIZES", on_host.SIZES + ("mx_attend_shared_workspace_size", "mx_lora_workspace_size",
                                                           "mx_logprobs_workspace_size"))
    return Machine(monkeypatch)


def zeros(*shape, dtype=BF16, card=0):
    return gpu(torch.zeros(*shape, dtype=dtype), card)


def table(b=2, cols=30, card=0):
    return zeros(b, cols, dtype=torch.int32, card=card)


def adapters(count=3, rank=16, k=256, n=64, dtype=BF16):
    return mx.Adapters(zeros(count, rank, k, dtype=dtype), zeros(count, n, rank, dtype=dtype), zeros(count, dtype=F32))


def shared(stream=None, **kw):
    a = dict(q=heads(2, 4), cache=cache(), prefix=ints(20), prefix_length=ints(1), page_table=table(), lengths=ints(2), lse=True)
    a.update(kw)
    return mx.mx_attend_shared(**a, stream=stream)


def read(stream=None, **kw):
    a = dict(cache=cache(), slots=ints(5, torch.int64))
    a.update(kw)
    return mx.mx_cache_read(**a, stream=stream)


def lora(stream=None, **kw):
    a = dict(x=zeros(4, 256), adapters=adapters(), ids=ints(4), base=zeros(4, 64))
    a.update(kw)
    return mx.mx_lora(**a, stream=stream)


def probs(stream=None, **kw):
    a = dict(logits=zeros(4, 90000), targets=ints(4, torch.int64), top=5)
    a.update(kw)
    return mx.mx_logprobs(**a, stream=stream)


def back(stream=None, **kw):
    a = dict(d_logprob=zeros(4, dtype=F32), d_entropy=zeros(4, dtype=F32), logits=zeros(4, 100), targets=ints(4, torch.int64),
             lse=zeros(4, dtype=F32), entropy=zeros(4, dtype=F32))
    a.update(kw)
    return mx.mx_logprobs_backward(**a, stream=stream)


CALLS = [shared, read, lora, probs, back]


@pytest.mark.parametrize("call", CALLS)
def test_streams(machine, call):
    check(machine, call)


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_given_by_name(machine, call):
    call(Stream(1))
    assert number(machine.launches[0][1][-1]) == 1


@pytest.mark.parametrize("call", CALLS)
def test_another_current_device(machine, call):
    machine.device = 1
    with pytest.raises(ValueError, match="device"):
        call()
    assert not machine.launches


def on(card, t):
    return gpu(t.clone(), card)


BAD = [
    (shared, dict(q=heads(2, 4, 32))), (shared, dict(q=on(1, heads(2, 4)))), (shared, dict(page_table=table(3))),
    (shared, dict(page_table=zeros(2, 30, dtype=torch.int64))), (shared, dict(page_table=table(card=1))),
    (shared, dict(page_table=zeros(30, 2, dtype=torch.int32).t())), (shared, dict(lengths=ints(3))),
    (shared, dict(lengths=ints(2, torch.int64))), (shared, dict(prefix=ints(20, torch.int64))), (shared, dict(prefix=table())),
    (shared, dict(prefix=ints(40)[::2])), (shared, dict(prefix=on(1, ints(20)))), (shared, dict(prefix_length=ints(2))),
    (shared, dict(prefix_length=ints(1, torch.int64))), (shared, dict(out=heads(2, 3))), (shared, dict(lse=zeros(2, 3, dtype=F32))),
    (shared, dict(lse=zeros(2, 4))), (shared, dict(workspace=on(1, zeros(100)))),
    (read, dict(slots=ints(5))), (read, dict(slots=on(1, ints(5, torch.int64)))), (read, dict(slots=ints(10, torch.int64)[::2])),
    (read, dict(k=heads(4, 2))), (read, dict(v=heads(5, 3))), (read, dict(k=on(1, heads(5, 2)))),
    (lora, dict(x=zeros(4, 248))), (lora, dict(x=zeros(4, 256, dtype=F32))), (lora, dict(x=on(1, zeros(4, 256)))),
    (lora, dict(x=zeros(256, 4).t())), (lora, dict(ids=ints(5))), (lora, dict(ids=ints(4, torch.int64))), (lora, dict(ids=on(1, ints(4)))),
    (lora, dict(base=zeros(4, 63))), (lora, dict(base=zeros(64, 4).t())), (lora, dict(base=on(1, zeros(4, 64)))),
    (lora, dict(y=zeros(3, 64))), (lora, dict(y=on(1, zeros(4, 64)))), (lora, dict(workspace=on(1, zeros(10000)))),
    (probs, dict(logits=zeros(4, 100, 2))), (probs, dict(logits=zeros(100, 4).t(), targets=ints(4, torch.int64))),
    (probs, dict(targets=ints(5, torch.int64))), (probs, dict(targets=ints(4))), (probs, dict(targets=on(1, ints(4, torch.int64)))),
    (probs, dict(top=65)), (probs, dict(top=-1)), (probs, dict(logits=zeros(4, 3), top=4)), (probs, dict(workspace=on(1, zeros(10)))),
    (back, dict(lse=zeros(5, dtype=F32))), (back, dict(lse=zeros(4))), (back, dict(entropy=None)), (back, dict(d_logprob=zeros(4, 1, dtype=F32))),
    (back, dict(d_logits=zeros(4, 101))), (back, dict(d_logits=zeros(4, 100, dtype=F32))), (back, dict(d_logits=on(1, zeros(4, 100)))),
    (back, dict(d_logits=zeros(100, 4).t())), (back, dict(d_entropy=on(1, zeros(4, dtype=F32)))),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(machine, i):
    call, kw = BAD[i]
    with pytest.raises(ValueError):
        call(**kw)
    assert not machine.launches


def test_types(machine):
    for call, kw in ((shared, dict(q=heads(2, 4, dtype=torch.float16))), (lora, dict(base=zeros(4, 64, dtype=torch.float16))),
                     (lora, dict(out_dtype=torch.float16)), (read, dict(out_dtype=torch.float16)),
                     (probs, dict(logits=zeros(4, 90000, dtype=torch.float16)))):
        with pytest.raises(TypeError):
            call(**kw)
    assert not machine.launches


def test_host_operands(machine):
    host = gpu(torch.zeros(4, 256, dtype=BF16), -1)
    with pytest.raises(ValueError):
        lora(x=host)
    with pytest.raises(ValueError):
        probs(logits=gpu(torch.zeros(4, 100, dtype=BF16), -1), targets=gpu(torch.zeros(4, dtype=torch.int64), -1))
    assert not machine.launches


@pytest.mark.parametrize("a,b,s", [
    ((3, 16, 256), (2, 64, 16), None), ((3, 16, 256), (3, 64, 8), None), ((16, 256), (64, 16), None), ((3, 16, 256), (3, 64, 16), (2,)),
])
def test_adapters(a, b, s):
    with pytest.raises(ValueError):
        mx.Adapters(zeros(*a), zeros(*b), None if s is None else zeros(*s, dtype=F32))
    with pytest.raises(ValueError):
        mx.Adapters(zeros(3, 16, 256), zeros(3, 64, 16, dtype=F32))
    with pytest.raises(ValueError):
        mx.Adapters(zeros(3, 16, 256), zeros(3, 16, 64).transpose(1, 2))
    with pytest.raises(ValueError):
        mx.Adapters(zeros(3, 16, 256), zeros(3, 64, 16), zeros(3))


def test_outputs_given_count_as_changed(machine):
    out, lse = heads(2, 4), zeros(2, 4, dtype=F32)
    k, y, dz = heads(5, 2), zeros(4, 64), zeros(4, 100)
    before = [t._version for t in (out, lse, k, y, dz)]
    shared(out=out, lse=lse), read(k=k), lora(y=y), back(d_logits=dz)
    assert [t._version for t in (out, lse, k, y, dz)] == [v + 1 for v in before]


def test_defaults(machine):
    assert lora(base=None).dtype == BF16 and lora(base=zeros(4, 64, dtype=F32)).dtype == F32
    assert read(v=heads(5, 2, dtype=F32))[0].dtype == F32
    assert len(probs(top=0)) == 3 and len(probs()) == 5
    assert back(d_logprob=None, d_entropy=None, entropy=None).shape == (4, 100)
