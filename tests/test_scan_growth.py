"""The selective scan with decays above one (A dt > 0), where the factor of a whole segment or chunk leaves fp32 although every
token's state and gradient stay inside it; against the recurrence token by token in 64 bits.  A token's factor is off by 2^-22 and
its exponent's rounding, half an ulp of at most 3: 3.2e-7 of it, and a value comes through at most 170 tokens of such: 5.4e-5; a
segment's sum of dt, up to 128, is rounded to 2^-18 by each of at most 84 additions: 3.2e-4 of the factor at worst.  Together 4e-4 of
a value whose terms have one sign (all but dy here); sums with dy of both signs get five times that of their largest value."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import mix

DEV = "cuda"
TOL = 4e-4


def draw(L, D, N, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(u=rnd(L, D).abs(), A=0.5 + 0.5 * torch.rand(D, N, generator=g), B=rnd(L, 1, N).abs(), C=rnd(L, 1, N).abs(),
                S0=torch.zeros(1, D, N), dy=rnd(L, D))


def ins(a, dev=None, dtype=None):
    t = [a[k] if dev is None else a[k].to(dev) for k in ("u", "delta", "A", "B", "C")]
    return [x if i == 2 or dev is None else x[None] for i, x in enumerate(t)] if dtype is None else [x.to(dtype) for x in t]


def forward(a):
    y, last = efla.efla_scan_fwd(*ins(a, DEV), S0=a["S0"].to(DEV), softplus=False)
    efla.efla_get_status()
    u, delta, A, B, C = ins(a, dtype=torch.float64)
    return (y[0].cpu(), last.cpu()), mix.scan_all([(0, len(u))], u, delta, A, B, C, None, None, None, a["S0"].double(), False)


def steps(L, *parts):
    """delta [L]: (from, value) pieces."""
    d = torch.zeros(L)
    for at, v in parts:
        d[at:] = v
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 8, 16, 64])
def test_forward_zero_state_through_growing_segments(N):
    """No input for most of the axis: zeros stay zeros, whatever a segment's tokens together would make of a state."""
    L, D = 700, 16
    a = draw(L, D, N, N)
    a["delta"] = steps(L, (0, 1.6))[:, None].expand(L, D) * (1 + 0.05 * torch.rand(L, D, generator=torch.Generator().manual_seed(1)))
    a["u"][:690] = 0
    for got, want in zip(*forward(a)):
        assert bool(torch.isfinite(got).all())
        assert bool(((got.double() - want).abs() <= TOL * want.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 8, 16, 64])
def test_forward_small_state_through_a_growing_segment(N):
    """A state of 1e-30 grows by up to 2^180 over the second segment's 80 tokens, and shrinks again."""
    L, D = 700, 16
    a = draw(L, D, N, N)
    a["delta"] = steps(L, (0, -0.001), (80, 1.5), (164, -1.5), (250, -0.1))[:, None].expand(L, D) * (1 + 0.02 * torch.rand(L, D, generator=torch.Generator().manual_seed(1)))
    a["u"][:164] = 0
    a["u"][164:] *= -1         # (dt u > 0 where dt < 0: every term has one sign)
    a["S0"] = 1e-30 * (1 + torch.rand(1, D, N, generator=torch.Generator().manual_seed(2)))
    for got, want in zip(*forward(a)):
        assert bool(torch.isfinite(got).all())
        assert bool(((got.double() - want).abs() <= TOL * want.abs()).all())


def backward(a):
    t = ins(a, DEV)
    got = efla.efla_scan_bwd(*t, a["dy"].to(DEV)[None], S0=a["S0"].to(DEV), softplus=False)
    efla.efla_get_status()
    u, delta, A, B, C = ins(a, dtype=torch.float64)
    args = [u, delta, A, B, C, None, None, None, a["S0"].double()]
    want = mix.grads(lambda *x: mix.scan_all([(0, len(u))], *x, False), args, a["dy"].double(), None)
    names = ("du", "ddelta", "dA", "dB", "dC", None, None, None, "dS0")
    return {n: (g.cpu().double().reshape(w.shape), w) for n, g, w in zip(names, got, want) if n}


def zeros_between(N):
    """32 ordinary tokens, 16 that empty the state, 80 that grow (what is) nothing, 32 ordinary ones without a gradient."""
    L, D = 160, 24
    a = draw(L, D, N, N)
    a["delta"] = steps(L, (0, 0.05), (32, -100.0), (48, 20.0), (128, -1.0))[:, None].expand(L, D).contiguous()
    a["u"][32:128] = 0
    a["dy"][32:] = 0
    return a


def small_values(N):
    """A state and gradients of 1e-30 that 32 tokens behind the first chunk grow by up to 2^138, forwards and backwards."""
    L, D = 128, 24
    a = draw(L, D, N, N)
    a["delta"] = steps(L, (0, -0.01), (32, 3.0), (64, -0.2))[:, None].expand(L, D) * (1 + 0.02 * torch.rand(L, D, generator=torch.Generator().manual_seed(1)))
    a["u"][:64] = 0
    a["dy"] *= 1e-30
    a["S0"] = 1e-30 * (1 + torch.rand(1, D, N, generator=torch.Generator().manual_seed(2)))
    return a


def close(name, got, want):
    assert bool(torch.isfinite(got).all()), name
    assert float((got - want).abs().max()) <= 5 * TOL * float(want.abs().max()), name


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 8, 16, 64])
def test_backward_states_through_growing_chunks(N):
    """dC is of the states alone."""
    got, want = backward(zeros_between(N))["dC"]
    close("dC", got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [4, 8, 16, 64])
@pytest.mark.parametrize("case", [zeros_between, small_values])
def test_backward_gradients_through_growing_chunks(case, N):
    for name, (got, want) in backward(case(N)).items():
        close(name, got, want)
