"""Which device the gated rule's and the norm's calls go to.  Stand-ins for tensors and the library: no GPU
needed, nothing is launched."""
import contextlib
import types

import pytest
import torch

import exact_flow_recurrence_gb300 as efla

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Fake:
    """What the binding asks of a dense CUDA tensor."""

    is_cuda = True

    def __init__(self, *shape, dtype=BF, device=1):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x7f0000000000

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


def fwd():
    a = dict(q=Fake(1, 1, 8, 16), k=Fake(1, 1, 8, 16), v=Fake(1, 2, 8, 16), g=Fake(1, 2, 8, dtype=F32), beta=Fake(1, 2, 8, dtype=F32),
             S0=Fake(1, 2, 16, 16, dtype=F32), o=Fake(1, 2, 8, 16), S_final=Fake(1, 2, 16, 16, dtype=F32),
             workspace=Fake(1 << 20, dtype=torch.uint8))
    return efla.efla_gated_fwd, a


def packed():
    a = {n: t if n in ("S0", "S_final", "workspace") else Fake(*t.shape[1:], dtype=t.dtype) for n, t in fwd()[1].items()}
    return efla.efla_gated_fwd, dict(a, offsets=Fake(2, dtype=I32))


def bwd():
    a = {n: t for n, t in fwd()[1].items() if n not in ("o", "S_final")}
    return efla.efla_gated_bwd, dict(a, dO=Fake(1, 2, 8, 16), dS_final=Fake(1, 2, 16, 16, dtype=F32), dq=Fake(1, 1, 8, 16),
                                     dk=Fake(1, 1, 8, 16), dv=Fake(1, 2, 8, 16))


def step():
    return efla.efla_gated_step, dict(q=Fake(1, 1, 16), k=Fake(1, 1, 16), v=Fake(1, 2, 16), g=Fake(1, 2, dtype=F32),
                                      beta=Fake(1, 2, dtype=F32), S=Fake(3, 2, 16, 16, dtype=F32), slots=Fake(1, dtype=I32),
                                      o=Fake(1, 2, 16))


def norm_fwd():
    return efla.efla_norm_fwd, dict(x=Fake(4, 64), weight=Fake(64, dtype=F32), bias=Fake(64, dtype=F32), y=Fake(4, 64),
                                    stats=Fake(4, 2, dtype=F32))


def norm_bwd():
    return efla.efla_norm_bwd, dict(x=Fake(4, 64), weight=Fake(64, dtype=F32), dy=Fake(4, 64), stats=Fake(4, 2, dtype=F32),
                                    workspace=Fake(1 << 24, dtype=torch.uint8))


CALLS = [fwd, packed, bwd, step, norm_fwd, norm_bwd]


@pytest.fixture()
def gpus(monkeypatch):
    """Device 0 is the current one; `seen` collects the device that each library call finds, and its stream."""
    state = types.SimpleNamespace(current=0, stream=None, seen=[])

    @contextlib.contextmanager
    def device(d):
        before, state.current = state.current, torch.device(d).index
        try:
            yield
        finally:
            state.current = before

    @contextlib.contextmanager
    def stream(s):
        before, state.stream = state.stream, s
        try:
            with device(s.device):
                yield
        finally:
            state.stream = before

    class Stream:
        def __init__(self, handle=0, device=None):
            self.cuda_stream, self.device = handle, torch.device("cuda", state.current) if device is None else device

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 256
            return lambda *a: state.seen.append((name, state.current, a[-1])) or 0

    monkeypatch.setattr(efla, "_plans", {})
    monkeypatch.setattr(efla, "load_library", Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream",
                        lambda i: 1000 * i + (state.stream.cuda_stream if state.stream else 0), raising=False)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=F32, device=None: empty(*shape, device=device) if str(device) == "meta"
                        else Fake(*(shape[0] if isinstance(shape[0], torch.Size) else shape), dtype=dtype, device=device.index))
    state.Stream = Stream
    return state


@pytest.mark.parametrize("call", CALLS)
def test_the_tensors_device_is_made_current(gpus, call):
    fn, a = call()
    fn(**a)
    assert gpus.seen == [(fn.__name__, 1, 1000)] and gpus.current == 0


@pytest.mark.parametrize("call", CALLS)
def test_streams_belong_to_the_tensors_device(gpus, call):
    fn, a = call()
    for s in (7, gpus.Stream(7, torch.device("cuda", 1)), types.SimpleNamespace(cuda_stream=7)):
        fn(**a, stream=s)
    assert gpus.seen == [(fn.__name__, 1, 1007)] * 3
    with pytest.raises(ValueError, match="stream"):
        fn(**a, stream=gpus.Stream(7, torch.device("cuda", 0)))
    assert gpus.current == 0 and len(gpus.seen) == 3


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in c()[1] if n not in ("v", "x")])
def test_tensors_of_another_device_are_refused(gpus, call, name):
    fn, a = call()
    for wrong in ("cuda", "cpu"):
        t = a[name]
        b = Fake(*t.shape, dtype=t.dtype, device=0)
        b.is_cuda = wrong == "cuda"
        with pytest.raises(ValueError, match=name):
            fn(**dict(a, **{name: b}))
    if call is step or call is fwd:   # (v itself)
        a["v"].is_cuda = False
        with pytest.raises(ValueError):
            fn(**a)
    assert gpus.seen == []
