"""Pins of the gated reference (oracle/gated.py) against facts that do not come from it: the
ungated C oracle at g = 0, decay alone at beta = 0, a hand-worked step, central differences."""
import math

import pytest
import torch

import oracle
from oracle import gated as og


def _draw(B, H, Hk, L, dk, dv, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    return (r(B, Hk, L, dk) / dk ** 0.5, r(B, Hk, L, dk) / dk ** 0.5, r(B, H, L, dv),
            -torch.nn.functional.softplus(r(B, H, L)), torch.sigmoid(r(B, H, L)), r(B, H, dk, dv), r(B, H, L, dv))


@pytest.mark.parametrize("exact", [False, True])
def test_no_decay_is_the_ungated_recurrence(exact):
    q, k, v, g, beta, S0, dO = _draw(2, 3, 3, 21, 16, 32)
    f = lambda x: x.float()  # noqa: E731
    q, k, v, beta, S0, dO = (f(x) for x in (q, k, v, beta, S0, dO))
    o, S = og.fwd(*(x.double() for x in (q, k, v, torch.zeros_like(beta), beta, S0)), exact=exact)
    o_ref, S_ref = oracle.fwd(q, k, v, beta, S0, euler=not exact)
    assert abs(o.numpy() - o_ref).max() < 1e-12 and abs(S.numpy() - S_ref).max() < 1e-12
    d = og.bwd(*(x.double() for x in (q, k, v, torch.zeros_like(beta), beta, dO, S0)), exact=exact)
    ref = oracle.bwd(q, k, v, beta, dO, S0, euler=not exact)
    for got, want in zip((d[0], d[1], d[2], d[4], d[5]), ref):
        assert abs(got.numpy() - want).max() < 1e-10


def test_decay_alone():
    q, k, v, g, beta, S0, _ = _draw(1, 2, 1, 9, 16, 16)
    _, S = og.fwd(q, k, v, g, torch.zeros_like(beta), S0)
    assert torch.allclose(S, S0 * g.sum(-1).exp()[..., None, None], rtol=1e-13)


def test_hand_worked_step():
    """dk = dv = 1: S = 2, f = 1/2, k = 3, v = 5, beta = 1/4 -> r = 5 - 3, S = 1 + 3/2, o = q S."""
    one = lambda x: torch.full((1, 1, 1, 1), x, dtype=torch.float64)  # noqa: E731
    o, S = og.fwd(one(2.), one(3.), one(5.), one(math.log(.5))[0], one(.25)[0], one(2.))
    assert abs(S.item() - 2.5) < 1e-15 and abs(o.item() - 5.0) < 1e-15


@pytest.mark.parametrize("exact", [False, True])
def test_gradients_against_differences(exact):
    x = list(_draw(1, 2, 1, 7, 4, 3, seed=3))
    dO, dS = x[6], torch.randn(1, 2, 4, 3, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
    grads = og.bwd(*x[:5], dO, x[5], dS, exact=exact)

    def loss(y):
        o, S = og.fwd(*y, exact=exact)
        return float((o * dO).sum() + (S * dS).sum())

    gen = torch.Generator().manual_seed(1)
    for n, d in enumerate(grads):
        for _ in range(4):
            i = int(torch.randint(x[n].numel(), (1,), generator=gen))
            ends = []
            for h in (1e-6, -1e-6):
                y = [t.clone() for t in x[:6]]
                y[n].view(-1)[i] += h
                ends.append(loss(y))
            assert abs((ends[0] - ends[1]) / 2e-6 - float(d.reshape(-1)[i])) < 1e-7 * (1 + abs(float(d.reshape(-1)[i])))


def test_norm_reference_against_brute_force():
    x, w, b = [1.0, 2.0, 4.0], [1.0, -1.0, 2.0], [0.0, 1.0, 0.5]
    m = sum(x) / 3
    s = 1 / math.sqrt(sum((t - m) ** 2 for t in x) / 3 + 0.1)
    y, st = og.norm_fwd(*(torch.tensor(t, dtype=torch.float64) for t in ([x], w, b)), 0.1)
    assert all(math.isclose(y[0, i], (x[i] - m) * s * w[i] + b[i], rel_tol=1e-13) for i in range(3))
    assert math.isclose(st[0, 0], m) and math.isclose(st[0, 1], s)
