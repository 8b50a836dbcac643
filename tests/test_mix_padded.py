"""Packed sequences on an axis that is longer than they are: what outputs hold at the tokens behind them (and in front) stays."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from test_devices import BF, Fake, gpus  # noqa: F401
from test_mix_devices import scan_bwd

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,G", [(16, 1), (5, 2), (32, 2), (4, 1)])
def test_gradients_of_a_padded_axis(N, G, dtype):
    """Every gradient of a token outside is zero where it was, the others as on an axis without padding."""
    T, D, ends = 200, 24, [9, 60, 60, 131]
    u, delta, z, dy = (torch.randn(T, D, device=DEV).to(dtype) for _ in range(4))
    B, C = (torch.randn(T, G, N, device=DEV).to(dtype) for _ in range(2))
    A = -torch.rand(D, N, device=DEV)
    off = lambda at: torch.tensor([e - at for e in ends], dtype=torch.int32, device=DEV)  # noqa: E731
    outs = {n: torch.zeros_like(t) for n, t in dict(du=u, ddelta=delta, dz=z, dB=B, dC=C).items()}
    got = efla.efla_scan_bwd(u, delta, A, B, C, dy, None, z, offsets=off(0), **outs)
    inner = [t[9:131] for t in (u, delta, B, C, dy, z)]
    want = efla.efla_scan_bwd(*inner[:2], A, *inner[2:5], None, inner[5], offsets=off(9))
    efla.efla_get_status()
    tol = 2.0 ** -7 if dtype == torch.bfloat16 else 1e-5     # (the chunks lie elsewhere: sums in another order, then half an ulp each)
    for name, p, q in zip(("du", "ddelta", "dA", "dB", "dC", None, "dz"), got, want):
        if name == "dA":
            assert float((p - q).abs().max()) <= 1e-5 * float(q.abs().max())
        elif name:
            assert p is outs[name]
            assert float(p[:9].abs().max()) == 0.0 and float(p[131:].abs().max()) == 0.0
            assert bool(((p[9:131].float() - q.float()).abs() <= tol * q.float().abs() + 1e-5 * float(q.float().abs().max())).all()), name


@pytest.mark.parametrize("name", ["dB", "dC"])
def test_gradients_of_another_shape_type_or_device_are_refused(gpus, name):  # noqa: F811
    fn, a = scan_bwd()
    fn(**a, **{name: Fake(2, 8, 1, 4)})
    assert len(gpus.seen) == 1
    for t in (Fake(2, 8, 1, 5), Fake(2, 8, 4), Fake(2, 8, 1, 4, dtype=torch.float32), Fake(2, 8, 1, 4, device=0)):
        with pytest.raises(ValueError, match=name):
            fn(**a, **{name: t})
    assert len(gpus.seen) == 1
