"""The gated rule where its calls are easiest to get wrong: tokens that a zero beta masks, keys and values
far from 1, tokens outside every packed sequence, more chunks than the gradient kernel has CTAs, and rows
between rows.  Bounds as in test_gated unless a test derives its own."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import gated as og
from parity import TOL_F32, assert_close
from test_gated import BF, DEV, F32, draw, gpu, ref64

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def run(x, mode, out_dtype=F32, **kw):
    y = gpu(x)
    a = [y[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = efla.efla_gated_fwd(*a, y["S0"], mode=mode, out_dtype=out_dtype, **kw)
    d = efla.efla_gated_bwd(*a, y["dO"], y["S0"], y["dS"], mode=mode, out_dtype=out_dtype, **kw)
    efla.efla_get_status()
    return o, S, d


@pytest.mark.parametrize("shape", [(1, 4, 2, 33, 64, 48), (2, 4, 2, 333, 128, 128), (3, 48, 24, 150, 96, 80),
                                   (1, 20, 20, 2100, 128, 128)])
def test_output_does_not_depend_on_the_state_asked_for(shape):
    """o of a call that returns no state is, bit for bit, o of the call that does."""
    y = gpu(draw(*shape, BF, efla.EULER, rate=0.05, seed=21))
    a = [y[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    for out in (BF, F32):
        with_state = efla.efla_gated_fwd(*a, out_dtype=out, path=efla.TENSOR)
        without = efla.efla_gated_fwd(*a, out_dtype=out, path=efla.TENSOR, want_state=False)
        efla.efla_get_status()
        assert without[1] is None and torch.equal(with_state[0], without[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", [efla.EULER, efla.EXACT])
@pytest.mark.parametrize("size", [1.0, 1e12])
def test_masked_tokens_of_any_size(size, mode, dtype):
    """beta = 0 masks a token: whatever its key and value (as long as products of keys are finite), the others'
    results are those of the definition, and so is its own beta's gradient."""
    x = draw(1, 4, 2, 200, 128, 64, dtype, mode, rate=0.1, seed=23)
    mask = torch.zeros(200, dtype=torch.bool)
    mask[[0, 20, 21, 22, 63, 64, 130, 199]] = True
    gen = torch.Generator().manual_seed(24)
    for n in ("k", "v"):
        x[n][:, :, mask] = (size * torch.randn(x[n][:, :, mask].shape, generator=gen)).to(dtype)
    x["beta"][:, :, mask] = 0.0
    o, S, d = run(x, mode)
    (o_ref, S_ref), g_ref = ref64(x, mode)
    assert_close("o", o, o_ref, TOL_F32)
    assert_close("S_final", S, S_ref, TOL_F32)
    for n, a, b in zip(GRADS, d, g_ref):
        if n == "dS0":
            assert_close(n, a, b, TOL_F32)
            continue
        assert_close(n, a[:, :, ~mask], b[:, :, ~mask], TOL_F32)
        if n in ("dk", "dv"):
            assert float(a[:, :, mask].abs().max()) == 0.0, n
        else:
            assert_close(n + " of the masked", a[:, :, mask], b[:, :, mask], TOL_F32)


@pytest.mark.parametrize("beta", [0.0, 1e-30])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_masked_tokens_at_scales(scale, beta):
    """beta's gradient where beta is zero or next to it, with values far from 1."""
    x = draw(1, 2, 2, 100, 128, 128, BF, efla.EULER, seed=25)
    x["v"], x["S0"] = (x["v"].float() * scale).to(BF), x["S0"] * scale
    x["dO"], x["dS"] = (x["dO"].float() / scale).to(BF), x["dS"] / scale
    x["beta"][:, :, 10:50] = beta
    d = run(x, efla.EULER)[2]
    for n, a, b in zip(GRADS, d, ref64(x, efla.EULER)[1]):
        assert_close(n, a, b, TOL_F32)
        if n == "dbeta":
            assert_close("dbeta of the masked", a[:, :, 10:50], b[:, :, 10:50], TOL_F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_keys_in_exact_mode(dtype):
    """||k||^2 about 1e26: alpha is 1 / ||k||^2, a projection, and stays one in the gradients."""
    x = draw(1, 2, 2, 150, 128, 128, dtype, efla.EXACT, rate=0.1, seed=26)
    x["k"][:, 0] = (x["k"][:, 0].float() * 2.0 ** 43).to(dtype)
    o, S, d = run(x, efla.EXACT)
    (o_ref, S_ref), g_ref = ref64(x, efla.EXACT)
    for h in (0, 1):   # (each head on the scale of its own)
        assert_close("o", o[:, h], o_ref[:, h], TOL_F32)
        assert_close("S_final", S[:, h], S_ref[:, h], TOL_F32)
        for n, a, b in zip(GRADS, d, g_ref):
            if n == "dbeta" and h == 0:   # e^{-beta ||k||^2} of it
                assert float(a[:, h].abs().max()) == 0.0
            elif n != "dk" or h == 1:
                assert_close(n, a[:, h], b[:, h], TOL_F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("power", [30, 43])
def test_key_gradient_of_long_keys_in_exact_mode(power, dtype):
    """dk through ||k||^2, where 1 / ||k||^4 is below what fp32 holds."""
    x = draw(1, 2, 2, 70, 128, 128, dtype, efla.EXACT, rate=0.1, seed=28)
    x["k"] = (x["k"].float() * 2.0 ** power).to(dtype)
    d = run(x, efla.EXACT)[2]
    assert_close("dk", d[1], ref64(x, efla.EXACT)[1][1], TOL_F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_fp32_gradients_carry_fp32(dtype):
    """dq and dk of an fp32 call, by the norm of their error: about eight products of up to 128 terms one
    after another, sqrt(128) 2^-24 each, are 2e-6 of the result (an operand of 17 bits would add 4e-6)."""
    x = draw(1, 2, 2, 200, 128, 128, dtype, efla.EULER, rate=0.1, seed=22)
    d = run(x, efla.EULER)[2]
    for n, a, b in zip(GRADS, d, ref64(x, efla.EULER)[1]):
        err = float((a.double().cpu() - b).norm() / b.norm())
        assert err <= 2e-6, (n, err)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ends", [[150, 250, 250, 391], [40, 41], [300, 300]])
def test_tokens_outside_every_sequence(ends, dtype):
    """Tokens before the first offset and behind the last: not read (they are NaN), not written."""
    H, Hk, dk, dv, T = 4, 2, 128, 64, 420
    x = draw(1, H, Hk, T, dk, dv, dtype, efla.EULER, seed=27, state=False)
    live = torch.zeros(T, dtype=torch.bool)
    live[ends[0]:ends[-1]] = True
    y = {n: t[0].clone() for n, t in x.items() if t is not None}
    for t in y.values():
        t[:, ~live] = float("nan")
    y = {n: t.to(DEV) for n, t in y.items()}
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    args = [y[n] for n in ("q", "k", "v", "g", "beta")]
    for out in (F32, BF):
        o, dq, dk_, dv_ = (torch.full_like(y[n], 7.0, dtype=out) for n in ("v", "q", "k", "v"))
        _, S = efla.efla_gated_fwd(*args, offsets=off, o=o, out_dtype=out)
        d = efla.efla_gated_bwd(*args, y["dO"], offsets=off, out_dtype=out, dq=dq, dk=dk_, dv=dv_)
        efla.efla_get_status()
        for n, t in (("o", o), ("dq", dq), ("dk", dk_), ("dv", dv_)):
            assert bool((t[:, ~live.to(DEV)] == 7.0).all()), n
        for b, (a, e) in enumerate(zip(ends, ends[1:])):
            if a == e:
                assert float(S[b].abs().max()) == 0.0
                continue
            s = {n: None if t is None else t[:, :, a:e] for n, t in x.items()}
            (o_ref, S_ref), g_ref = ref64(s, efla.EULER)
            assert_close("o", o[None, :, a:e], o_ref, TOL_F32, stored_bf16=out == BF)
            assert_close("S_final", S[b:b + 1], S_ref, TOL_F32)
            for n, got, want in zip(GRADS[:5], d, g_ref):
                assert_close(n, got[None, :, a:e], want, TOL_F32, stored_bf16=got.dtype == BF)


def gpu64(x, mode):
    """The reference on the GPU (fp64 too), for sizes that take the CPU too long."""
    y = {n: t.to(DEV).double() for n, t in x.items()}
    a, e = [y[n] for n in ("q", "k", "v", "g", "beta")], mode == efla.EXACT
    return og.fwd(*a, y["S0"], exact=e), og.bwd(*a, y["dO"], y["S0"], y["dS"], exact=e)


@pytest.mark.parametrize("mode,shape", [(efla.EULER, (4, 32, 32, 130, 128, 128)), (efla.EXACT, (10, 16, 8, 260, 128, 128)),
                                        (efla.EULER, (1, 8, 8, 2600, 64, 96)), (efla.EXACT, (6, 32, 8, 333, 128, 64))])
def test_more_chunks_than_ctas(mode, shape):
    """The gradient kernel's CTAs, one an SM, take several chunks each: q and k again, sums over value heads
    again, outputs in place of the operands before."""
    B, _, Hk, L = shape[:4]
    assert B * -(-L // 64) * Hk > 2 * 152 or Hk < shape[1]
    x = draw(*shape, BF, mode, rate=0.1, seed=29, token_first=L % 2 == 1)
    (o_ref, S_ref), g_ref = gpu64(x, mode)
    for out in (F32, BF):
        o, S, d = run(x, mode, out)
        assert_close("o", o, o_ref, TOL_F32, stored_bf16=out == BF)
        assert_close("S_final", S, S_ref, TOL_F32)
        for n, a, b in zip(GRADS, d, g_ref):
            assert_close(n, a, b, TOL_F32, stored_bf16=a.dtype == BF)


@pytest.mark.parametrize("H,Hk", [(8, 8), (16, 8)])
def test_more_packed_chunks_than_ctas(H, Hk):
    """The same with ragged, single-token and empty sequences between full chunks."""
    ends = [0, 130, 130, 131, 700, 1341, 1405, 2300, 2300, 3001]
    B, T, dk, dv = len(ends) - 1, ends[-1], 128, 128
    assert (T // 64 + B) * Hk > 304
    x = draw(1, H, Hk, T, dk, dv, BF, efla.EULER, rate=0.1, seed=30, token_first=True, state=False)
    gen = torch.Generator().manual_seed(31)
    S0, dS = (0.3 * torch.randn(B, H, dk, dv, generator=gen) for _ in range(2))
    y = {n: t.to(DEV)[0] for n, t in x.items() if t is not None}
    args = [y[n] for n in ("q", "k", "v", "g", "beta")]
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    for out in (F32, BF):
        d = efla.efla_gated_bwd(*args, y["dO"], S0.to(DEV), dS.to(DEV), offsets=off, out_dtype=out)
        efla.efla_get_status()
        for b, (a, e) in enumerate(zip(ends, ends[1:])):
            if a == e:
                assert torch.equal(d[5][b].cpu(), dS[b])
                continue
            s = {n: t[:, :, a:e] for n, t in x.items() if t is not None}
            s["S0"], s["dS"] = S0[b:b + 1], dS[b:b + 1]
            want = gpu64(s, efla.EULER)[1]
            for n, got, ref in zip(GRADS[:5], d, want):
                assert_close(n, got[None, :, a:e], ref, TOL_F32, stored_bf16=got.dtype == BF)
            assert_close("dS0", d[5][b:b + 1], want[5], TOL_F32)


def inside(shape, dtype, pad):
    """A strided view in the middle of a buffer of sevens, `pad` elements between its rows, and the buffer."""
    buf = torch.full((shape[0] + 2, *shape[1:-1], shape[-1] + pad), 7.0, dtype=dtype, device=DEV)
    return buf[1:-1][..., :shape[-1]], buf


def untouched(view, buf):
    """Every element of the buffer outside the view is still seven, and none inside is NaN."""
    w = buf.clone()
    w[1:-1][..., :view.shape[-1]] = 7.0
    return bool((w == 7.0).all()) and not bool(view.isnan().any())


@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(2, 2, 1, 33, 64, 48), (2, 4, 2, 150, 128, 80)])
def test_nothing_is_written_around_the_outputs(shape, dtype, pad):
    """o, dq, dk, dv, states and the norm's outputs as views: what lies around and between their rows stays."""
    B, H, Hk, L, dk, dv = shape
    x = draw(*shape, dtype, efla.EULER, seed=32)
    (o_ref, S_ref), _ = ref64(x, efla.EULER)
    x = gpu(x)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o = inside((B, H, L, dv), dtype, pad)
    Sbuf = torch.full((B + 2, H, dk, dv), 7.0, device=DEV)
    S = Sbuf[1:-1]
    efla.efla_gated_fwd(*a, x["S0"], o=o[0], S_final=S)
    d = [inside(t.shape, dtype, pad) for t in (x["q"], x["k"], x["v"])]
    efla.efla_gated_bwd(*a, x["dO"], x["S0"], x["dS"], dq=d[0][0], dk=d[1][0], dv=d[2][0])
    efla.efla_get_status()
    assert untouched(*o) and all(untouched(*t) for t in d)
    assert bool((Sbuf[0] == 7).all()) and bool((Sbuf[-1] == 7).all())
    assert_close("o", o[0], o_ref, TOL_F32, stored_bf16=dtype == BF)
    assert_close("S_final", S, S_ref, TOL_F32)
    # the step, on the states in the middle of their buffer
    po = inside((B, H, dv), dtype, pad)
    efla.efla_gated_step(*(t[:, :, 0] for t in a), S, o=po[0])
    efla.efla_get_status()
    assert untouched(*po) and bool((Sbuf[0] == 7).all()) and bool((Sbuf[-1] == 7).all())


@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_is_written_around_the_norm(dtype, pad):
    y, ybuf = inside((70, 264), dtype, pad)
    x = torch.randn(70, 264, device=DEV).to(dtype)
    sbuf = torch.full((72, 2), 7.0, device=DEV)
    efla.efla_norm_fwd(x, torch.ones(264, device=DEV), y=y, stats=sbuf[1:-1])
    efla.efla_get_status()
    assert untouched(y, ybuf) and bool((sbuf[0] == 7).all()) and bool((sbuf[-1] == 7).all())
    assert not bool((sbuf[1:-1] == 7).any())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 2, 2, 1, 64, 64), (3, 2, 1, 2, 128, 64), (1, 2, 2, 70, 64, 128)])
def test_gate_gradients_under_strong_decay(shape, dtype):
    """Gates that forget nearly everything at every token (e^-15 and less) have gradients that small: what does
    not decay is in none of the sums that make them, so each is right on its own scale."""
    x = draw(*shape, dtype, efla.EULER, seed=33)
    gen = torch.Generator().manual_seed(34)
    x["g"] = -(15.0 + 3.0 * torch.rand(x["g"].shape, generator=gen))
    for n, a, b in zip(GRADS, run(x, efla.EULER)[2], ref64(x, efla.EULER)[1]):
        assert_close(n, a, b, TOL_F32)
