"""Which device the convolution's, the scan's and the RMS norm's calls go to.  Stand-ins for tensors and the library: no GPU
needed, nothing is launched."""
import types

import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from test_devices import BF, F32, I32, Fake, gpus  # noqa: F401


def conv_fwd():
    return efla.efla_conv_fwd, dict(x=Fake(2, 8, 16), weight=Fake(16, 4, dtype=F32), bias=Fake(16, dtype=F32), S0=Fake(2, 3, 16),
                                    y=Fake(2, 8, 16), S_final=Fake(2, 3, 16))


def conv_packed():
    fn, a = conv_fwd()
    return fn, dict(a, x=Fake(8, 16), y=Fake(8, 16), offsets=Fake(3, dtype=I32))


def conv_bwd():
    return efla.efla_conv_bwd, dict(x=Fake(2, 8, 16), weight=Fake(16, 4, dtype=F32), dy=Fake(2, 8, 16), bias=Fake(16, dtype=F32),
                                    S0=Fake(2, 3, 16), dS_final=Fake(2, 3, 16), dx=Fake(2, 8, 16), workspace=Fake(1 << 20, dtype=torch.uint8))


def conv_step():
    return efla.efla_conv_step, dict(x=Fake(2, 16), weight=Fake(16, 4, dtype=F32), S=Fake(5, 3, 16), bias=Fake(16, dtype=F32),
                                     slots=Fake(2, dtype=I32), y=Fake(2, 16))


def scan_fwd():
    return efla.efla_scan_fwd, dict(u=Fake(2, 8, 16), delta=Fake(2, 8, 16), A=Fake(16, 4, dtype=F32), B=Fake(2, 8, 1, 4), C=Fake(2, 8, 1, 4),
                                    D=Fake(16, dtype=F32), z=Fake(2, 8, 16), delta_bias=Fake(16, dtype=F32), S0=Fake(2, 16, 4, dtype=F32),
                                    y=Fake(2, 8, 16), S_final=Fake(2, 16, 4, dtype=F32), workspace=Fake(1 << 20, dtype=torch.uint8))


def scan_packed():
    fn, a = scan_fwd()
    cut = {n: Fake(*a[n].shape[1:]) for n in ("u", "delta", "z", "y", "B", "C")}
    return fn, dict(a, **cut, offsets=Fake(3, dtype=I32))


def scan_bwd():
    a = {n: t for n, t in scan_fwd()[1].items() if n not in ("y", "S_final")}
    return efla.efla_scan_bwd, dict(a, dy=Fake(2, 8, 16), dS_final=Fake(2, 16, 4, dtype=F32), du=Fake(2, 8, 16), ddelta=Fake(2, 8, 16),
                                    dz=Fake(2, 8, 16))


def scan_step():
    return efla.efla_scan_step, dict(u=Fake(2, 16), delta=Fake(2, 16), A=Fake(16, 4, dtype=F32), B=Fake(2, 1, 4), C=Fake(2, 1, 4),
                                     S=Fake(5, 16, 4, dtype=F32), D=Fake(16, dtype=F32), z=Fake(2, 16), delta_bias=Fake(16, dtype=F32),
                                     slots=Fake(2, dtype=I32), y=Fake(2, 16))


def rms_fwd():
    return efla.efla_rms_fwd, dict(x=Fake(4, 256), weight=Fake(256, dtype=F32), residual=Fake(4, 256), y=Fake(4, 256), h=Fake(4, 256),
                                   rstd=Fake(4, dtype=F32))


def rms_quant():
    fn, a = rms_fwd()
    return fn, dict(a, y=Fake(4, 256, dtype=torch.float8_e4m3fn), scale=Fake(4, 2, dtype=F32), group=128)


def rms_bwd():
    return efla.efla_rms_bwd, dict(h=Fake(4, 256), weight=Fake(256, dtype=F32), dy=Fake(4, 256), rstd=Fake(4, dtype=F32), dh=Fake(4, 256),
                                   dx=Fake(4, 256), workspace=Fake(1 << 20, dtype=torch.uint8))


CALLS = [conv_fwd, conv_packed, conv_bwd, conv_step, scan_fwd, scan_packed, scan_bwd, scan_step, rms_fwd, rms_quant, rms_bwd]
FIRST = ("x", "u", "h")


@pytest.mark.parametrize("call", CALLS)
def test_the_tensors_device_is_made_current(gpus, call):  # noqa: F811
    fn, a = call()
    fn(**a)
    assert gpus.seen == [(fn.__name__, 1, 1000)] and gpus.current == 0


@pytest.mark.parametrize("call", CALLS)
def test_streams_belong_to_the_tensors_device(gpus, call):  # noqa: F811
    fn, a = call()
    for s in (7, gpus.Stream(7, torch.device("cuda", 1)), types.SimpleNamespace(cuda_stream=7)):
        fn(**a, stream=s)
    assert gpus.seen == [(fn.__name__, 1, 1007)] * 3
    with pytest.raises(ValueError, match="stream"):
        fn(**a, stream=gpus.Stream(7, torch.device("cuda", 0)))
    assert gpus.current == 0 and len(gpus.seen) == 3


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n, t in c()[1].items()
                                       if isinstance(t, Fake) and n != list(c()[1])[0]])
def test_tensors_of_another_device_shape_or_type_are_refused(gpus, call, name):  # noqa: F811
    fn, a = call()
    t = a[name]
    for wrong in ("cuda", "cpu"):
        b = Fake(*t.shape, dtype=t.dtype, device=0)
        b.is_cuda = wrong == "cuda"
        with pytest.raises(ValueError, match=name):
            fn(**dict(a, **{name: b}))
    if name != "workspace":
        wrong = [Fake(*t.shape, dtype=torch.float64)] if name not in ("weight", "bias") else []
        if name not in ("weight", "A", "C", "offsets"):     # (those that say the sizes)
            wrong.append(Fake(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype))
        for b in wrong:
            with pytest.raises((ValueError, TypeError)):
                fn(**dict(a, **{name: b}))
    assert gpus.seen == []
