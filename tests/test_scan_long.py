"""The selective scan where a CTA walks many tiles forward and several chunks backward, against the recurrence token by token in
64 bits.  max |err| / rms <= 2.5e-4: a decay e^x is off by (2.3 |x| + 5) 2^-24 at most and 2e-8 on average, so that a state which
remembers m tokens is off by m 2e-8 + sqrt(m) 1e-7 of itself, 2.4e-5 at the m <= 1000 met here, and the largest value of an output
is up to ten times its rms; the gradients of A and of the bias weigh a state by both and get twice that.  Values stored in bf16 add
half an ulp."""
import math
import random

import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from parity import assert_close

TOL = 2.5e-4
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
NAMES = ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "dbias", "dS0")


def recurrence(u, delta, A, B, C, D, z, bias, S0, dy, dS, softplus=True):
    """y, S_final and the gradients in NAMES' order, of [B, L, ...] in the inputs' type (fp64), a token at a time."""
    nb, L, Di = u.shape
    rep = Di // B.shape[2]
    bm, c = (t.repeat_interleave(rep, 2) for t in (B, C))
    raw = delta if bias is None else delta + bias
    dt = torch.nn.functional.softplus(raw, threshold=80) if softplus else raw
    sig = None if z is None else torch.sigmoid(z)
    gy = dy if z is None else dy * z * sig
    hs, h = [], S0
    for t in range(L):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * u[:, t])[..., None] * bm[:, t]
        hs.append(h)
    o = torch.stack([(hs[t] * c[:, t]).sum(-1) for t in range(L)], 1) + D * u
    y = o if z is None else o * z * sig
    q, dA = dS, torch.zeros_like(A)
    du, ddt, db, dc = [], [], [], []
    for t in range(L - 1, -1, -1):
        p = q + gy[:, t, :, None] * c[:, t]
        dc.append((hs[t] * gy[:, t, :, None]).unflatten(1, (-1, rep)).sum(2))
        db.append((p * (dt[:, t] * u[:, t])[..., None]).unflatten(1, (-1, rep)).sum(2))
        s1 = (p * bm[:, t]).sum(-1)
        q = p * torch.exp(dt[:, t, :, None] * A)
        e = q * (hs[t - 1] if t else S0)
        dA += (dt[:, t, :, None] * e).sum(0)
        du.append(dt[:, t] * s1)
        ddt.append((A * e).sum(-1) + u[:, t] * s1)
    du, ddt, db, dc = (torch.stack(x[::-1], 1) for x in (du, ddt, db, dc))
    ddelta = ddt * torch.sigmoid(raw) if softplus else ddt
    return y, h, (du + D * gy, ddelta, dA, db, dc, (gy * u).sum((0, 1)), None if z is None else dy * o * sig * (1 + z * (1 - sig)),
                  None if bias is None else ddelta.sum((0, 1)), q)


def make(B, L, D, N, G, dtype, gate=True, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + D + 17 * N + L)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    size = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=g, device=DEV))
    return dict(u=rnd(B, L, D).to(dtype), delta=(0.5 * rnd(B, L, D)).to(dtype), A=-(1 + torch.arange(N, device=DEV)) * torch.exp(0.1 * rnd(D, N)),
                B=rnd(B, L, G, N).to(dtype), C=rnd(B, L, G, N).to(dtype), D=1 + 0.1 * rnd(D), z=rnd(B, L, D).to(dtype) if gate else None,
                bias=size + torch.log(-torch.expm1(-size)), S0=0.5 * rnd(B, D, N), dy=rnd(B, L, D).to(dtype), dS=0.1 * rnd(B, D, N))


TOKENS = ("u", "delta", "B", "C", "z", "dy")


def compare(y, last, got, ref_y, ref_last, ref, bf):
    assert_close("y", y, ref_y, TOL, stored_bf16=bf)
    assert_close("S_final", last, ref_last, TOL)
    for name, p, r in zip(NAMES, got, ref):
        if r is None:
            assert p is None, name
            continue
        assert_close(name, p, r, (2 if name in ("dA", "dbias") else 1) * TOL, stored_bf16=bf and name in ("du", "ddelta", "dB", "dC", "dz"))


def calls(a, off=None):
    ins, rest = [a[k] for k in ("u", "delta", "A", "B", "C")], [a[k] for k in ("D", "z", "bias", "S0")]
    y, last = efla.efla_scan_fwd(*ins, *rest, offsets=off)
    got = efla.efla_scan_bwd(*ins, a["dy"], *rest, a["dS"], offsets=off)
    again = efla.efla_scan_fwd(*ins, *rest, offsets=off) + efla.efla_scan_bwd(*ins, a["dy"], *rest, a["dS"], offsets=off)
    efla.efla_get_status()
    assert all(p is q or torch.equal(p, q) for p, q in zip((y, last) + got, again))
    return y, last, got


def d64(a):
    return {k: None if t is None else t.double() for k, t in a.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,D,N,G,gate", [(8, 1024, 2048, 16, 1, True), (4, 1024, 2048, 16, 1, True), (8, 700, 1000, 32, 2, False), (6, 517, 2050, 8, 1, True),
                                            (5, 403, 3000, 4, 3, False), (4, 301, 1111, 13, 1, True), (3, 260, 1100, 64, 1, False)])
def test_many_tiles_and_chunks(B, L, D, N, G, gate, dtype):
    """Forward without segments (96 CTAs and more: 64 tiles of 16 tokens, 44, 17) and in a few; backward with two to 14 chunks a CTA;
    ragged ends."""
    a = make(B, L, D, N, G, dtype, gate)
    compare(*calls(a), *recurrence(**d64(a)), dtype == BF)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,N,G", [(1000, 32, 2), (2048, 16, 1), (515, 8, 1)])
def test_packed_many_chunks(D, N, G, dtype):
    """Some 5000 tokens on one axis, sequences that end at every place of a chunk; each by itself is the reference."""
    r = random.Random(D)
    lens = [601, 0, 1, 33, 5] + [r.randint(0, 70) for _ in range(25)] + [1023, 32, 31, 64, 0] + [r.randint(1, 6) for _ in range(20)] + [1009, 512]
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    T, n = ends[-1], len(lens)
    a = make(1, T, D, N, G, dtype)
    g = torch.Generator(device=DEV).manual_seed(1)
    a.update({k: a[k][0] for k in TOKENS}, S0=0.5 * torch.randn(n, D, N, generator=g, device=DEV), dS=0.1 * torch.randn(n, D, N, generator=g, device=DEV))
    y, last, got = calls(a, torch.tensor(ends, dtype=torch.int32, device=DEV))
    b, parts = d64(a), []
    total = [torch.zeros_like(b[k]) for k in ("A", "D", "bias")]
    for i, (s, e) in enumerate(zip(ends, ends[1:])):
        one = {k: t[None, s:e] if k in TOKENS else t[i:i + 1] if k in ("S0", "dS") else t for k, t in b.items()}
        if e == s:
            parts.append((one["u"], one["S0"], (one["u"], one["u"], 0, one["B"], one["C"], 0, one["u"], 0, one["dS"])))
            continue
        parts.append(recurrence(**one))
        for t, j in zip(total, (2, 5, 7)):
            t += parts[-1][2][j]
    of = lambda j: torch.cat([p[2][j][0] for p in parts])  # noqa: E731
    ref = (of(0), of(1), total[0], of(3), of(4), total[1], of(6), total[2], torch.cat([p[2][8] for p in parts]))
    compare(y, last, got, torch.cat([p[0][0] for p in parts]), torch.cat([p[1] for p in parts]), ref, dtype == BF)
