"""The gated delta rule's entry points on the GPU against the token-by-token fp64 reference.

Tolerances (max |err| / rms), fixed from the arithmetic: a chunk's result passes through about
eight products of up to 128 terms.  On the fp32 cores each contributes about sqrt(128) 2^-24 =
7e-7 of the result's rms; on the tensor cores the computed operands are sums of two bf16 parts,
2^-18 to 2^-17 of the operand, about 4e-6 after the same chain.  Five standard deviations over
the elements of a tensor give 3e-5 and 2e-5 more for cancelling sums: 1e-4, the framework's
bound for fp32 work.  Values stored in bf16 add half an ulp (parity.assert_close).
"""
import itertools

import numpy as np
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import gated as og
from parity import TOL_F32, assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def draw(B, H, Hk, L, dk, dv, dtype, mode, rate=0.3, seed=0, token_first=False, state=True):
    """Inputs on the CPU as the GPU gets them: [B,heads,L,d] views, stored head- or token-major."""
    gen = torch.Generator().manual_seed(seed)

    def r(heads, *d):
        x = torch.randn(B, L, heads, *d, generator=gen) if token_first else torch.randn(B, heads, L, *d, generator=gen)
        return x.transpose(1, 2) if token_first else x

    k = r(Hk, dk)
    k = k / k.norm(dim=-1, keepdim=True).clamp_min(1e-9)
    if mode == efla.EXACT:
        k = k * torch.exp(0.5 * r(Hk, 1))
    x = dict(q=(r(Hk, dk) / dk ** 0.5).to(dtype), k=k.to(dtype), v=r(H, dv).to(dtype),
             g=-rate * torch.nn.functional.softplus(r(H)), beta=torch.sigmoid(r(H)), dO=r(H, dv).to(dtype))
    x["S0"] = 0.3 * torch.randn(B, H, dk, dv, generator=gen) if state else None
    x["dS"] = 0.3 * torch.randn(B, H, dk, dv, generator=gen) if state else None
    return x


def gpu(x):
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def ref64(x, mode):
    f = [None if x[n] is None else x[n].double() for n in ("q", "k", "v", "g", "beta", "dO", "S0", "dS")]
    q, k, v, g, beta, dO, S0, dS = f
    e = mode == efla.EXACT
    return og.fwd(q, k, v, g, beta, S0, exact=e), og.bwd(q, k, v, g, beta, dO, S0, dS, exact=e)


def check_fwd(x, mode, path=efla.AUTO, out_dtype=None, want=None, **kw):
    y = gpu(x)
    o, S = efla.efla_gated_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["S0"], mode=mode, path=path,
                               out_dtype=out_dtype, **kw)
    efla.efla_get_status()
    o_ref, S_ref = (want or ref64(x, mode))[0]
    assert_close("o", o, o_ref, TOL_F32, stored_bf16=o.dtype == BF)
    assert_close("S_final", S, S_ref, TOL_F32)
    return o, S


def check_bwd(x, mode, path=efla.AUTO, out_dtype=None, want=None):
    y = gpu(x)
    d = efla.efla_gated_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["dO"], y["S0"], y["dS"], mode=mode, path=path,
                            out_dtype=out_dtype)
    efla.efla_get_status()
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), d, (want or ref64(x, mode))[1]):
        assert_close(n, a, b, TOL_F32, stored_bf16=a.dtype == BF)
    return d


SHAPES = [  # B, H, Hk, L, dk, dv
    (1, 1, 1, 1, 16, 16), (2, 2, 1, 3, 16, 32), (1, 2, 2, 31, 48, 80), (1, 3, 3, 32, 64, 64), (2, 4, 2, 33, 128, 48),
    (1, 2, 1, 63, 128, 128), (1, 1, 1, 64, 128, 128), (2, 2, 2, 65, 128, 128), (1, 4, 1, 150, 96, 112),
    (3, 2, 2, 200, 128, 64), (1, 2, 1, 321, 128, 128)]


@pytest.mark.parametrize("mode", [efla.EULER, efla.EXACT])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_both_directions(shape, dtype, mode):
    x = draw(*shape, dtype, mode, seed=sum(shape), token_first=shape[3] % 2 == 1)
    want = ref64(x, mode)
    check_fwd(x, mode, out_dtype=F32, want=want)
    check_bwd(x, mode, out_dtype=F32, want=want)
    if dtype == BF:
        check_fwd(x, mode, want=want)
        check_bwd(x, mode, want=want)
        if shape[3] in (33, 65, 150):
            check_fwd(x, mode, efla.SIMT, want=want)
            check_bwd(x, mode, efla.SIMT, want=want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rate", [0.0, 1e-3, 4.0, 60.0])
def test_decay_rates(rate, dtype):
    """No decay at all, slow, and decays that wipe the state within a token (sums of thousands)."""
    x = draw(1, 2, 2, 140, 128, 128, dtype, efla.EULER, rate=rate, seed=5)
    want = ref64(x, efla.EULER)
    check_fwd(x, efla.EULER, out_dtype=F32, want=want)
    check_bwd(x, efla.EULER, out_dtype=F32, want=want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_reset_gates(dtype):
    """g = -inf, and the type's lowest value, forget the state: tokens before do not reach those after,
    and no inf - inf is formed."""
    x = draw(1, 2, 1, 130, 64, 64, dtype, efla.EULER, seed=6)
    for t, low in ((0, -float("inf")), (40, -float("inf")), (41, torch.finfo(F32).min), (100, -float("inf"))):
        x["g"][:, :, t] = low
    want = ref64(x, efla.EULER)
    o, _ = check_fwd(x, efla.EULER, out_dtype=F32, want=want)
    d = check_bwd(x, efla.EULER, out_dtype=F32, want=want)
    assert float(d[5].abs().max()) == 0.0     # the initial state is forgotten at once
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["v"][:, :, :41] = 1.0
    o2, _ = efla.efla_gated_fwd(*(gpu(y)[n] for n in ("q", "k", "v", "g", "beta", "S0")), out_dtype=F32)
    assert torch.equal(o[:, :, 41:], o2[:, :, 41:])


def test_zero_and_hard_keys():
    """Zero keys and queries, beta 0 and 1, repeated keys (the chunk's inverse at its worst)."""
    for dtype in (BF, F32):
        x = draw(1, 2, 2, 128, 128, 128, dtype, efla.EXACT, rate=0.0, seed=8)
        x["k"][:, 0, 10:20] = 0
        x["q"][:, 0, 5:9] = 0
        x["k"][:, 1, 1:] = x["k"][:, 1, :1]
        x["beta"][:, :, 30:60] = 1.0
        x["beta"][:, :, 60:70] = 0.0
        for mode in (efla.EXACT, efla.EULER):
            if mode == efla.EULER:   # unit keys: beta ||k||^2 stays within the stable range
                x["k"] = (x["k"].float() / x["k"].float().norm(dim=-1, keepdim=True).clamp_min(1e-9)).to(dtype)
            want = ref64(x, mode)
            check_fwd(x, mode, out_dtype=F32, want=want)
            check_bwd(x, mode, out_dtype=F32, want=want)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_scales(scale):
    """Values far from 1: no operand format narrows the range (bf16 parts keep fp32's exponents)."""
    x = draw(1, 2, 2, 100, 128, 128, BF, efla.EULER, seed=9)
    x["v"], x["S0"] = (x["v"].float() * scale).to(BF), x["S0"] * scale
    x["dO"], x["dS"] = (x["dO"].float() / scale).to(BF), x["dS"] / scale
    want = ref64(x, efla.EULER)
    check_fwd(x, efla.EULER, out_dtype=F32, want=want)
    check_bwd(x, efla.EULER, out_dtype=F32, want=want)


ENDS = [[0, 1], [0, 0, 5, 5, 70], [0, 64, 128, 129, 129, 300], [0, 200, 201, 265, 266, 266, 397]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ends", ENDS)
@pytest.mark.parametrize("token_first", [False, True])
def test_packed_sequences(ends, dtype, token_first):
    """Sequences of any lengths on one axis, as if each were alone; a NaN in one stays in it."""
    H, Hk, dk, dv = 4, 2, 128, 64
    B, T = len(ends) - 1, ends[-1]
    x = draw(1, H, Hk, T, dk, dv, dtype, efla.EULER, seed=T, token_first=token_first, state=False)
    gen = torch.Generator().manual_seed(1)
    S0, dS = (0.3 * torch.randn(B, H, dk, dv, generator=gen) for _ in range(2))
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    y = {n: t.to(DEV)[0] for n, t in x.items() if t is not None}
    args = [y[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = efla.efla_gated_fwd(*args, S0.to(DEV), offsets=off, out_dtype=F32)
    d = efla.efla_gated_bwd(*args, y["dO"], S0.to(DEV), dS.to(DEV), offsets=off, out_dtype=F32)
    efla.efla_get_status()
    for b, (a, e) in enumerate(zip(ends, ends[1:])):
        if a == e:
            assert torch.equal(S[b].cpu(), S0[b]) and torch.equal(d[5][b].cpu(), dS[b])
            continue
        s = {n: t[:, :, a:e] for n, t in x.items() if t is not None}
        s["S0"], s["dS"] = S0[b:b + 1], dS[b:b + 1]
        (o_ref, S_ref), g_ref = ref64(s, efla.EULER)
        assert_close("o", o[None, :, a:e], o_ref, TOL_F32)
        assert_close("S_final", S[b:b + 1], S_ref, TOL_F32)
        for n, got, want in zip(("dq", "dk", "dv", "dg", "dbeta"), d, g_ref):
            assert_close(n, got[None, :, a:e], want, TOL_F32)
        assert_close("dS0", d[5][b:b + 1], g_ref[5], TOL_F32)
    hurt = max(range(B), key=lambda b: ends[b + 1] - ends[b])
    a, e = ends[hurt], ends[hurt + 1]
    for n in ("q", "k", "v", "dO", "g", "beta"):
        z = dict(y)
        z[n] = z[n].clone()
        z[n][:, a:e] = float("nan")
        args = [z[m] for m in ("q", "k", "v", "g", "beta")]
        o2, S2 = efla.efla_gated_fwd(*args, S0.to(DEV), offsets=off, out_dtype=F32)
        d2 = efla.efla_gated_bwd(*args, z["dO"], S0.to(DEV), dS.to(DEV), offsets=off, out_dtype=F32)
        efla.efla_get_status()
        keep = torch.ones(T, dtype=torch.bool)
        keep[a:e] = False
        for p, r in [(o, o2)] + list(zip(d[:5], d2[:5])):
            assert torch.equal(p[:, keep.to(DEV)], r[:, keep.to(DEV)]), n
        rest = [b for b in range(B) if b != hurt]
        assert torch.equal(S[rest], S2[rest]) and torch.equal(d[5][rest], d2[5][rest]), n


def test_clamped_offsets():
    """Offsets outside the axis (device data) are clamped, not followed."""
    x = gpu(draw(1, 2, 2, 90, 64, 64, BF, efla.EULER, seed=3, state=False))
    args = [x[n][0] for n in ("q", "k", "v", "g", "beta")]
    good = torch.tensor([0, 30, 90], dtype=torch.int32, device=DEV)
    wild = torch.tensor([-7, 30, 1 << 30], dtype=torch.int32, device=DEV)
    a, b = (efla.efla_gated_fwd(*args, offsets=o) for o in (good, wild))
    efla.efla_get_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_fused_projection_slices(dtype):
    """q, k, v as slices of one [B, L, width] projection, and dq, dk, dv into slices of one gradient
    buffer, equal the dense calls; an odd element offset (no 16-byte rows) gives the same numbers to
    rounding."""
    B, H, Hk, L, dk, dv = 2, 4, 2, 100, 64, 64
    x = gpu(draw(B, H, Hk, L, dk, dv, dtype, efla.EULER, seed=4, token_first=True))
    sizes = [Hk * dk, Hk * dk, H * dv]
    dense = efla.efla_gated_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S0"], out_dtype=F32)
    dgrad = efla.efla_gated_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["dO"], x["S0"], x["dS"], out_dtype=F32)
    for shift in (0, 8, 1):
        def sliced(buf):
            return [c.unflatten(-1, (h, d)).transpose(1, 2) for c, h, d in
                    zip(buf[..., shift:shift + sum(sizes)].split(sizes, -1), (Hk, Hk, H), (dk, dk, dv))]
        buf = torch.empty(B, L, sum(sizes) + 16, dtype=dtype, device=DEV)
        q, k, v = sliced(buf)
        for a, n in ((q, "q"), (k, "k"), (v, "v")):
            a.copy_(x[n])
        o, S = efla.efla_gated_fwd(q, k, v, x["g"], x["beta"], x["S0"], out_dtype=F32)
        grads = sliced(torch.full(buf.shape, 7.0, dtype=F32, device=DEV))
        d = efla.efla_gated_bwd(q, k, v, x["g"], x["beta"], x["dO"], x["S0"], x["dS"], out_dtype=F32, dq=grads[0], dk=grads[1],
                                dv=grads[2])
        efla.efla_get_status()
        for a, b in [(o, dense[0]), (S, dense[1])] + list(zip(d, dgrad)):
            assert_close("slice", a, b.double().cpu().numpy(), TOL_F32 if shift == 1 else 1e-12)


def test_broadcast_inputs():
    """Stride-0 inputs (one beta and one query for all heads) equal their copies."""
    x = gpu(draw(2, 4, 4, 70, 64, 64, BF, efla.EULER, seed=5))
    beta, q = x["beta"][:, :1].expand(2, 4, 70), x["q"][:, :1].expand(2, 4, 70, 64)
    a = efla.efla_gated_fwd(q, x["k"], x["v"], x["g"], beta, x["S0"], out_dtype=F32)
    b = efla.efla_gated_fwd(q.contiguous(), x["k"], x["v"], x["g"], beta.contiguous(), x["S0"], out_dtype=F32)
    efla.efla_get_status()
    for s, t in zip(a, b):
        assert_close("broadcast", s, t.double().cpu().numpy(), TOL_F32)


def test_no_decay_matches_the_ungated_kernels():
    x = gpu(draw(1, 2, 2, 130, 128, 128, BF, efla.EXACT, rate=0.0, seed=11))
    o, S = efla.efla_gated_fwd(x["q"], x["k"], x["v"], torch.zeros_like(x["g"]), x["beta"], x["S0"], mode=efla.EXACT, out_dtype=F32)
    o2, S2 = efla.efla_fwd(x["q"], x["k"], x["v"], x["beta"], x["S0"], out_dtype=F32, path=efla.SIMT)
    efla.efla_get_status()
    assert_close("o", o, o2.double().cpu().numpy(), TOL_F32)
    assert_close("S", S, S2.double().cpu().numpy(), TOL_F32)


def test_repeatable_and_split():
    """Bitwise equal runs; a sequence in two calls equals one call (state handed on, in place)."""
    x = gpu(draw(2, 4, 2, 333, 128, 128, BF, efla.EULER, seed=12))
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = efla.efla_gated_fwd(*a, x["S0"], out_dtype=F32)
    o2, S2 = efla.efla_gated_fwd(*a, x["S0"], out_dtype=F32)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    d, d2 = (efla.efla_gated_bwd(*a, x["dO"], x["S0"], x["dS"]) for _ in range(2))
    assert all(torch.equal(p, r) for p, r in zip(d, d2))
    state = x["S0"].clone()
    parts = []
    for lo, hi in ((0, 100), (100, 333)):
        p, _ = efla.efla_gated_fwd(*(t[:, :, lo:hi] for t in a), state, S_final=state, out_dtype=F32)
        parts.append(p)
    efla.efla_get_status()
    assert_close("o", torch.cat(parts, 2), o.double().cpu().numpy(), TOL_F32)
    assert_close("S", state, S.double().cpu().numpy(), TOL_F32)


def test_gradients_against_differences():
    """Directional differences of the GPU forward itself (fp32): (f(x + h u) - f(x - h u)) / 2h against
    <grad, u>.  h = 1e-2 of unit-rms directions: truncation ~ h^2, rounding ~ 1e-6 |f| / h ~ 1e-3."""
    x = gpu(draw(1, 2, 1, 48, 32, 32, F32, efla.EXACT, seed=13))
    names = ("q", "k", "v", "g", "beta", "S0")
    d = efla.efla_gated_bwd(*(x[n] for n in names[:5]), x["dO"], x["S0"], x["dS"], mode=efla.EXACT)
    gen = torch.Generator(device=DEV).manual_seed(2)

    def loss(y):
        o, S = efla.efla_gated_fwd(*(y[n] for n in names), mode=efla.EXACT)
        return float((o.double() * x["dO"].double()).sum() + (S.double() * x["dS"].double()).sum())

    for n, grad in zip(names, d):
        u = torch.randn(x[n].shape, generator=gen, device=DEV)
        h = 1e-2 * float(x[n].square().mean().sqrt()) / x[n].numel() ** 0.5
        f = [loss({**x, n: x[n] + s * h * u}) for s in (1, -1)]
        got, want = (f[0] - f[1]) / (2 * h), float((grad.double() * u.double()).sum())
        scale = float(grad.double().norm() * u.double().norm()) / u.numel() ** 0.5
        assert abs(got - want) <= 2e-2 * max(abs(want), scale), (n, got, want)


def test_capture_and_other_stream():
    """A captured call replays; a call on a stream of its own equals the default one."""
    x = gpu(draw(2, 2, 2, 200, 128, 128, BF, efla.EULER, seed=14))
    a = [x[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    want = efla.efla_gated_fwd(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = efla.efla_gated_fwd(*a, stream=side)
    gd = efla.efla_gated_bwd(*a[:5], x["dO"], x["S0"], x["dS"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    wd = efla.efla_gated_bwd(*a[:5], x["dO"], x["S0"], x["dS"])
    assert all(torch.equal(p, r) for p, r in itertools.chain(zip(want, got), zip(wd, gd)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = efla.efla_gated_fwd(*a)
        capd = efla.efla_gated_bwd(*a[:5], x["dO"], x["S0"], x["dS"])
    for t in cap + capd:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    efla.efla_get_status()
    assert all(torch.equal(p, r) for p, r in itertools.chain(zip(want, cap), zip(wd, capd)))


# ------------------------------------------------------------------ the decode step
@pytest.mark.parametrize("mode", [efla.EULER, efla.EXACT])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (3, 4, 2, 48, 80), (2, 6, 3, 128, 128), (40, 8, 4, 128, 128),
                                   (5, 2, 1, 128, 96), (70, 16, 16, 128, 128), (3, 3, 3, 64, 128),
                                   (60, 8, 4, 112, 64), (80, 4, 4, 48, 128)])
def test_step(shape, dtype, mode):
    B, H, Hk, dk, dv = shape
    gen = torch.Generator().manual_seed(B)
    n = B + 3
    S = 0.3 * torch.randn(n, H, dk, dv, generator=gen)
    place = torch.randperm(n, generator=gen)[:B].to(torch.int32)
    if B > 2:
        place[1], place[2] = -1, n          # two sequences without a place
    live = [b for b in range(B) if 0 <= int(place[b]) < n]
    Sg, Sp = S.to(DEV), S[:B].to(DEV)
    R, Rp = S.double(), S[:B].double()
    for t in range(3):
        x = draw(B, H, Hk, 1, dk, dv, dtype, mode, seed=100 * B + t, state=False)
        f = [x[m].double() for m in ("q", "k", "v", "g", "beta")]
        a = [x[m][:, :, 0].to(DEV) for m in ("q", "k", "v", "g", "beta")]
        o = efla.efla_gated_step(*a, Sg, slots=place.to(DEV), mode=mode, out_dtype=F32)
        op = efla.efla_gated_step(*a, Sp, mode=mode)
        efla.efla_get_status()
        o_ref, new = og.fwd(*(y[live] for y in f), R[place[live].long()], exact=mode == efla.EXACT)
        R[place[live].long()] = new
        assert_close("o", o[live], o_ref[:, :, 0], TOL_F32)
        for b in range(B):
            if b not in live:
                assert float(o[b].abs().max()) == 0.0
        o_ref, Rp = og.fwd(*f, Rp, exact=mode == efla.EXACT)
        assert_close("o, no slots", op, o_ref[:, :, 0], TOL_F32, stored_bf16=dtype == BF)
    assert_close("S", Sg, R, TOL_F32)
    assert_close("S, no slots", Sp, Rp, TOL_F32)
    untouched = [i for i in range(n) if i not in place[live].tolist()]
    assert torch.equal(Sg[untouched].cpu(), S[untouched])


def test_step_strided_inputs_and_reset():
    """q, k, v as slices of one projection row (also at odd offsets); g = -inf starts from nothing."""
    B, H, dk, dv = 5, 4, 128, 128
    gen = torch.Generator().manual_seed(3)
    for shift in (0, 1):
        row = torch.randn(B, H * (2 * dk + dv) + 8, generator=gen).to(BF).to(DEV)
        q, k, v = (c.unflatten(-1, (H, d)) for c, d in
                   zip(row[:, shift:shift + H * (2 * dk + dv)].split([H * dk, H * dk, H * dv], -1), (dk, dk, dv)))
        k = k * 0.1
        g, beta = torch.full((B, H), -float("inf"), device=DEV), torch.full((B, H), 0.5, device=DEV)
        S = torch.randn(B, H, dk, dv, generator=gen).to(DEV)
        o = efla.efla_gated_step(q, k, v, g, beta, S, out_dtype=F32)
        efla.efla_get_status()
        want = 0.5 * k.double()[..., None] * v.double()[..., None, :]
        assert_close("S", S, want.cpu(), TOL_F32)
        assert_close("o", o, torch.einsum("bhkv,bhk->bhv", want, q.double()).cpu(), TOL_F32)


def test_steps_follow_the_chunked_pass():
    """Prefill by chunks, then decode token by token, equals the whole sequence at once."""
    x = gpu(draw(2, 4, 2, 90, 128, 128, BF, efla.EULER, seed=15))
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = efla.efla_gated_fwd(*a, x["S0"], out_dtype=F32)
    _, state = efla.efla_gated_fwd(*(t[:, :, :70] for t in a), x["S0"], out_dtype=F32)
    for t in range(70, 90):
        p = efla.efla_gated_step(*(y[:, :, t] for y in a), state, out_dtype=F32)
        assert_close("o", p, o[:, :, t].double().cpu().numpy(), TOL_F32)
    efla.efla_get_status()
    assert_close("S", state, S.double().cpu().numpy(), TOL_F32)


def test_binding_checks():
    x = gpu(draw(1, 2, 2, 8, 16, 16, BF, efla.EULER))
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError):
        efla.efla_gated_fwd(a[0], a[1], a[2], a[3].to(BF), a[4])
    with pytest.raises(ValueError):
        efla.efla_gated_fwd(a[0][:, :, :7], *a[1:])
    with pytest.raises(ValueError):
        efla.efla_gated_fwd(a[0].transpose(2, 3), a[1].transpose(2, 3).contiguous().transpose(2, 3), *a[2:])
    with pytest.raises(ValueError):
        efla.efla_gated_fwd(*a, x["S0"].double())
    with pytest.raises(ValueError):
        efla.efla_gated_step(*(t[:, :, 0] for t in a), x["S0"], slots=torch.zeros(1, device=DEV))
    with pytest.raises(efla.EflaError):
        efla.efla_gated_fwd(*a, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_empty():
    for L, B in ((0, 2), (5, 0)):
        x = gpu(draw(B, 2, 2, L, 32, 32, BF, efla.EULER))
        a = [x[n] for n in ("q", "k", "v", "g", "beta")]
        o, S = efla.efla_gated_fwd(*a, x["S0"])
        d = efla.efla_gated_bwd(*a, x["dO"], x["S0"], x["dS"])
        efla.efla_get_status()
        assert o.shape == x["v"].shape and torch.equal(S, x["S0"]) and torch.equal(d[5], x["dS"])


def test_large_strides():
    """Element offsets past 2^31: two sequences whose batch stride is 2^31 + 64 elements apart."""
    L, d = 70, 64
    big = torch.zeros((1 << 31) + 64 + 4 * L * d, dtype=BF, device=DEV)
    x = draw(2, 1, 1, L, d, d, BF, efla.EULER, seed=16, state=False)
    st = ((1 << 31) + 64, L * d, d, 1)
    views = {n: torch.as_strided(big, (2, 1, L, d), st, i * L * d) for i, n in enumerate(("q", "k", "v"))}
    for n, t in views.items():
        t.copy_(x[n])
    o, S = efla.efla_gated_fwd(views["q"], views["k"], views["v"], x["g"].to(DEV), x["beta"].to(DEV), out_dtype=F32)
    efla.efla_get_status()
    (o_ref, S_ref), _ = ref64(x, efla.EULER)
    assert_close("o", o, o_ref, TOL_F32)
    assert_close("S", S, S_ref, TOL_F32)
