"""How far a decay, a softplus and a sigmoid are off, as the header says.  In units of 2^-24 of the result: ex2.approx 4 (2^-22), its
exponent x log2(e) |x| for each rounding of it (one; two for a decay, whose A log2(e) is rounded first) and 0.22 |x| for the constant's
own; behind it a sigmoid has a sum (1), a reciprocal (2) and here a product (1), a softplus three roundings and a fit of 1.2e-8
(0.2), and a decay the 1.1e-8 that evens out the instruction's mean."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla

DEV = "cuda"


def off(got, want):
    """In units of 2^-24 of what is wanted."""
    return ((got.double() - want) / want).abs() * 2.0 ** 24


def line(lo, hi, n=1 << 20):
    g = torch.Generator(device=DEV).manual_seed(0)
    return lo + (hi - lo) * torch.rand(n // 64, 64, generator=g, device=DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(-86, -16), (-16, -1), (-1, 1), (1, 30)])
def test_sigmoid(lo, hi):
    x = line(lo, hi)
    w = torch.zeros(64, 2, device=DEV)
    w[:, 1] = 1
    y = efla.efla_conv_fwd(x[None], w, want_state=False)[0][0]
    efla.efla_get_status()
    d = x.double()
    assert bool((off(y, d * torch.sigmoid(d)) <= 1.3 * d.abs() + 8).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(-86, -16), (-16, -1), (-1, 1), (1, 30)])
def test_softplus(lo, hi):
    """The step of a scan without memory whose B, C and u are one: y = dt."""
    x = line(lo, hi)
    one = torch.ones(len(x), 1, 1, device=DEV)
    S = torch.zeros(len(x), 64, 1, device=DEV)
    y = efla.efla_scan_step(torch.ones_like(x), x, torch.zeros(64, 1, device=DEV), one, one, S)
    efla.efla_get_status()
    d = x.double()
    want = torch.log1p(torch.exp(-d.abs())) + d.clamp_min(0)
    assert bool((off(y, want) <= 1.3 * d.abs() + 8).all()) and torch.equal(S[..., 0], y)


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(-80, -8), (-8, -1), (-1, -0.125), (-0.125, -1e-3), (-1e-3, -1e-6), (0.01, 8)])
def test_decay(lo, hi):
    """A state of one through a token without input."""
    x = line(lo, hi)
    A = -torch.exp(2 * torch.randn(64, 1, generator=torch.Generator().manual_seed(1))).to(DEV)
    dt = x / A[:, 0]
    S = torch.ones(len(x), 64, 1, device=DEV)
    bc = torch.ones(len(x), 1, 1, device=DEV)
    efla.efla_scan_step(torch.zeros_like(x), dt, A, bc, bc, S, softplus=False)
    efla.efla_get_status()
    d = dt.double() * A[:, 0].double()
    got, want = S[..., 0], torch.exp(d)
    assert bool((off(got, want) <= 2.3 * d.abs() + 5).all())
    # the constant log2(e) in fp32 is 1.335e-8 of itself too small, the same way in every value: its part of the mean is 1.335e-8 |x|
    mean = float(((got.double() - want) / want).mean())
    assert abs(mean) <= (2e-8 if abs(lo) <= 0.125 else 5e-8) + 1.34e-8 * float(d.abs().mean())
