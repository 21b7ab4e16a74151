"""What the binding does on the host around a call: the streams on which it
converts and allocates, the sizes it hands to the library, the device it asks.
The library and the device are stand-ins, so none of it needs a GPU."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch
from torch.overrides import TorchFunctionMode

from compressed_sparse_long_hca_b200 import api


class FakeStream:
    def __init__(self, name):
        self.name, self.cuda_stream, self.device, self.waited = name, 16, torch.device("cuda", 0), []

    def wait_stream(self, other):
        self.waited.append(other.name)


class Streams(TorchFunctionMode):
    """Host tensors stand in for CUDA tensors (what is moved to "cuda", and
    what comes of that); every operation that would launch or allocate is
    noted with the stream that is current for it."""

    def __init__(self):
        super().__init__()
        self.current = FakeStream("current")
        self.work, self.cuda, self.kept, self.recorded = [], set(), [], []

    def on_cuda(self, t):
        self.kept.append(t)                    # (an id stays its own)
        self.cuda.add(id(t))
        return t

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def __torch_function__(self, func, types, args=(), kwargs=None):
        kwargs = kwargs or {}
        name = getattr(func, "__name__", "")
        if func == torch.Tensor.is_cuda.__get__:
            return id(args[0]) in self.cuda
        there = any(id(a) in self.cuda for a in args)
        if name == "to" and str(args[1]).startswith("cuda"):
            args, there = (args[0], "cpu"), True
            out = args[0].clone()
        else:
            out = func(*args, **kwargs)
        if name in ("to", "contiguous", "empty") and (there or name == "empty"):
            self.work.append((name, self.current.name))
        return self.on_cuda(out) if isinstance(out, torch.Tensor) and there else out


@pytest.fixture
def streams(monkeypatch):
    m = Streams()

    class Lib:
        @staticmethod
        def csa_gemm_fp8_quant_weight(*args):
            m.work.append(("kernel", "side" if args[-1] else "current"))
            return 0

    monkeypatch.setattr(api._lib, "load", lambda: Lib)
    monkeypatch.setattr(api, "_on_device", lambda index, call, *args: call(*args))
    monkeypatch.setattr(api, "_raw_stream", lambda stream, index: None if stream is None else stream.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: m.current)
    monkeypatch.setattr(torch.cuda, "stream", m.stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: m.recorded.append((id(t), s.name)))
    return m


@pytest.mark.parametrize("where", ["host array", "host tensor", "device tensor"])
def test_a_weight_is_quantised_on_one_stream(streams, where):
    """The conversion to BF16, the outputs' memory and the kernel belong to
    one stream, and a given one waits for the current one first."""
    a = np.ones((130, 256), np.float32)
    for stream, name in ((None, "current"), (FakeStream("side"), "side")):
        w = a if where == "host array" else torch.from_numpy(a.copy())
        if where == "device tensor":
            streams.on_cuda(w)
        streams.work.clear()
        with streams:
            codes, scales = api.quantize_fp8_weight(w, stream=stream)
        assert tuple(codes.shape) == (130, 256) and tuple(scales.shape) == (2, 2)
        assert [n for n, _ in streams.work].count("empty") == 2 and ("to", name) in streams.work
        assert streams.work[-1] == ("kernel", name)
        assert {s for _, s in streams.work} == {name}, streams.work
        if stream is not None:
            assert stream.waited == ["current"]
            assert (id(w), "side") in streams.recorded or where != "device tensor"
