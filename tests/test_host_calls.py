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
        if func == torch.Tensor.device.__get__ and id(args[0]) in self.cuda:
            return torch.device("cuda", 0)
        there = any(id(a) in self.cuda for a in args)
        if name == "empty":
            there, kwargs = str(kwargs["device"]).startswith("cuda"), {**kwargs, "device": "cpu"}
        if name == "to" and str(args[1]).startswith("cuda"):
            args, there = (args[0], "cpu"), True
            out = args[0].clone()
        else:
            out = func(*args, **kwargs)
        if name in ("to", "contiguous", "empty") and there:
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


@pytest.mark.parametrize("stream", [None, FakeStream("side")])
def test_a_weight_is_quantised_on_a_cuda_device_alone(streams, stream):
    """Nothing is launched for host memory, nor on another device's stream."""
    a = np.ones((8, 16), np.float32)
    with streams:
        with pytest.raises(ValueError, match="device"):
            api.quantize_fp8_weight(a, device="cpu", stream=stream)
        if stream is not None:
            with pytest.raises(ValueError, match="device"):
                api.quantize_fp8_weight(a, device="cuda:1", stream=stream)
    assert not streams.work


def _short_view():
    """100 bytes that end before the next 256-byte boundary."""
    buf = torch.zeros(1024, dtype=torch.uint8)
    skip = -buf.data_ptr() % 256 + 1
    return buf[skip: skip + 100]


class Sizes:
    """A library that needs 512 bytes of scratch and notes the size it is given (the argument at `place`)."""

    def __init__(self, **place):
        self.place, self.got = place, None

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *args: 512

        def call(*args):
            self.got = ctypes.c_size_t(args[self.place[name]]).value
            return 0
        return call


@pytest.mark.parametrize("entry", ["index_topk", "prefill_chunk", "Linear", "LinearFP8"])
def test_a_workspace_shorter_than_its_alignment_counts_nothing(monkeypatch, entry):
    """The library then refuses the call: no size wraps around."""
    monkeypatch.setattr(api, "_need", lambda *args, **kw: None)
    monkeypatch.setattr(api, "_stream", lambda stream: None)
    monkeypatch.setattr(api, "_raw_stream", lambda stream, index: None)
    monkeypatch.setattr(api, "_on_device", lambda index, call, *args: call(*args))
    ws, f = _short_view(), torch.float32
    lib = Sizes(csa_index_topk=12, csa_prefill_chunk=18, csa_gemm_bf16=9, csa_gemm_fp8=9)
    if entry in ("index_topk", "prefill_chunk"):
        c = object.__new__(api.Cache)
        c.handle, c.lib, c.n_csa, c.H, c.D, c.H_I, c.d_I, c.qdtype = None, lib, 1, 1, 8, 1, 32, torch.bfloat16
        ids, t = torch.zeros(1, dtype=torch.int32), torch.zeros
        if entry == "index_topk":
            c.index_topk(0, ids, t(1, 1, 32), t(1, 1), t(1, 128), ids, 4, ids, workspace=ws)
        else:
            c.prefill_chunk(0, ids, t(1, 2, 8), t(1, 2, 8), t(1, 2, 32), t(1, 2, 32), t(1, 2, 1, 8), t(1, 2, 1, 32), t(1, 2, 1), 4,
                            t(1), t(1, 2, 1, 8), workspace=ws)
    else:
        lin = object.__new__(getattr(api, entry))
        lin.lib, lin.n_out, lin.k_in, lin.groups, lin.device, lin._index, lin._need_bytes = lib, 4, 8, 1, ws.device, -1, {}
        lin.packed = torch.zeros(8, dtype=torch.uint8)
        lin(torch.zeros((20, 8), dtype=torch.bfloat16), torch.zeros((20, 4), dtype=f), workspace=ws)
    assert lib.got == 0


def test_device_errors_are_read_where_the_weight_is(monkeypatch):
    asked = []

    class Lib:
        @staticmethod
        def csa_gemm_check_device_error(stream):
            return 0

    monkeypatch.setattr(api._lib, "load", lambda: Lib)
    monkeypatch.setattr(api, "_on_device", lambda index, call, *args: asked.append((index, *args)) or call(*args))
    monkeypatch.setattr(api, "_raw_stream", lambda stream, index: ("current", index) if stream is None else stream.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_stream", lambda stream: ("current", 0) if stream is None else stream.cuda_stream)
    lin, side = object.__new__(api.LinearFP8), FakeStream("side")
    lin._index, side.device = 3, torch.device("cuda", 2)
    lin.check_device_error()
    lin.check_device_error(side)
    api.LinearFP8.check_device_error()
    api.LinearFP8.check_device_error(side)
    assert asked == [(3, ("current", 3)), (3, 16), (0, ("current", 0)), (2, 16)]


def test_projections_with_a_norm_refuse_bad_positions_before_the_first_launch():
    """The products would overwrite the outputs, which stay without their norm."""
    n, d, D, H, d_c = 3, 16, 8, 2, 16
    norm = object.__new__(api.HeadNorm)
    norm.dim, norm.rope, norm.rotate_k, norm._index, norm.device = D, 4, False, -1, torch.device("cpu")
    norm._q_weight = norm._k_weight = 0
    launched = []
    P = object.__new__(api.LayerProjections)
    P.csa, P.norm = False, norm
    P.W1 = P.W2 = lambda *args, **kw: launched.append(args)
    outs = dict(c=torch.zeros(n, 1, D), z=torch.zeros(n, 1, D), c_q=torch.zeros(n, d_c, dtype=torch.bfloat16),
                q=torch.zeros(n, H, D, dtype=torch.bfloat16))
    h = torch.zeros(n, d, dtype=torch.bfloat16)
    for bad in (None, torch.zeros(n), torch.zeros(n + 1, dtype=torch.int64), torch.zeros((n, 1), dtype=torch.int64)):
        with pytest.raises(ValueError, match="positions"):
            P(h, outs, positions=bad)
    with pytest.raises(ValueError, match="q must be"):
        P(h, {**outs, "q": outs["q"][:, :, :4]}, positions=torch.zeros(n, dtype=torch.int64))
    assert not launched
