"""The Python binding without a GPU: host tensors that say they lie on one, the
library's launches recorded instead of made, and streams that are names.  What
the library computes on the host alone (sizes) stays its own."""
import contextlib

import torch

import microscaling_block_quantization_amd as mx

SIZES = ("mx_query_sizes", "mx_qsnr_workspace_size", "mx_qk_rope_workspace_size", "mx_attend_workspace_size", "mx_status_string")


class Stream:
    def __init__(self, number, device=0):
        self.cuda_stream, self.device_index, self.device = number, device, torch.device("cuda", device)

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on `card`; remembers the stream it was
    allocated under and the streams its use was recorded on."""
    card = 0
    now = None                                     # the Machine whose streams count

    @property
    def is_cuda(self):
        return self.card >= 0

    def get_device(self):
        return self.card

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", ()) + (stream.cuda_stream,)

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if kwargs.get("device") is not None:
            kwargs["device"] = "cpu"
        out = super().__torch_function__(func, types, args, kwargs)
        if isinstance(out, torch.Tensor) and func in (torch.Tensor.new_empty, torch.empty_like):
            out.card = args[0].card
            cls.now.made(out)
        return out


def gpu(t, card=0):
    t = t.as_subclass(OnGpu)
    if card:
        t.card = card
    return t


class Machine:
    """One process with a current device and a current stream."""

    def __init__(self, monkeypatch):
        self.stream, self.device = Stream(1), 0
        self.launches, self.allocated = [], {}     # (name, args); address -> (stream, tensor)
        real = mx.lib()
        machine = self

        class Library:
            def __getattr__(self, name):
                if name in SIZES:
                    return getattr(real, name)
                return lambda *args: machine.launches.append((name, args)) or mx.MX_OK

        library = Library()
        monkeypatch.setattr(mx, "lib", lambda: library)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stream)
        monkeypatch.setattr(torch.cuda, "stream", self.under)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: self.stream.cuda_stream)
        monkeypatch.setattr(OnGpu, "now", self)
        make = torch.empty

        def empty(*args, device=None, **kw):
            return self.made(gpu(make(*args, **kw)))

        monkeypatch.setattr(torch, "empty", empty)

    @contextlib.contextmanager
    def under(self, stream):
        before = self.stream, self.device
        self.stream, self.device = stream, stream.device_index
        yield
        self.stream, self.device = before

    def made(self, t):
        self.allocated[t.data_ptr()] = (self.stream.cuda_stream, t)
        return t
