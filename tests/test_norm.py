"""Layer norm on the GPU against the fp64 reference (max |err| / rms <= 1e-5: sums of up to 16384
fp32 terms in trees, about log2(D) 2^-24 each, and 2^-24 a multiply; values stored in bf16 add half
an ulp; the weight's gradient adds rows / CTAs terms one after another, sqrt(rows) 2^-24 at most)."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import gated as og
from parity import assert_close

TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def _check(rows, D, dtype, wdtype, bias, pad=0, shift=0.0, eps=1e-5, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, D + pad, generator=gen) * 2 + shift).to(dtype)[:, :D]
    dy = torch.randn(rows, D + pad, generator=gen).to(dtype)[:, :D]
    w = (1 + 0.2 * torch.randn(D, generator=gen)).to(wdtype)
    b = (0.2 * torch.randn(D, generator=gen)).to(wdtype) if bias else None
    xg, dyg = (torch.empty(rows, D + pad, dtype=dtype, device=DEV)[:, :D].copy_(t) for t in (x, dy))
    bg = None if b is None else b.to(DEV)
    y, st = efla.efla_norm_fwd(xg, w.to(DEV), bg, eps=eps)
    y_ref, st_ref = og.norm_fwd(x.double(), w.double(), None if b is None else b.double(), eps)
    # the mean's error is measured against the row's deviation too: a mean near zero has no scale of its own
    assert float((st.cpu().double() - st_ref)[:, 0].abs().max()) <= TOL * float(x.double().abs().max())
    assert_close("rstd", st[:, 1], st_ref[:, 1], TOL * (1 + abs(shift)))
    assert_close("y", y, y_ref, TOL * (1 + abs(shift)), stored_bf16=dtype == BF)
    dx, dw, db = efla.efla_norm_bwd(xg, w.to(DEV), dyg, st, want_bias=bias)
    efla.efla_get_status()
    ref = og.norm_bwd(x.double(), w.double(), dy.double(), eps)
    # dx is a difference of terms of the size of rstd w dy: where it cancels (D = 2, where it is
    # eps / var of them) its error is measured against the terms, else the two scales agree
    terms = float((st_ref[:, 1:] * w.double() * dy.double()).square().mean().sqrt())
    scale = max(1.0, terms / float(ref[0].square().mean().sqrt())) if D == 2 else 1.0
    assert_close("dx", dx, ref[0], scale * TOL * (1 + abs(shift)), stored_bf16=dtype == BF)
    assert_close("dw", dw, ref[1], 2 * TOL * (1 + abs(shift)), stored_bf16=wdtype == BF)
    if bias:
        assert_close("db", db, ref[2], 2 * TOL, stored_bf16=wdtype == BF)
    else:
        assert db is None
    again = efla.efla_norm_bwd(xg, w.to(DEV), dyg, st, want_bias=bias)
    assert all(torch.equal(p, r) for p, r in zip((dx, dw), again))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,D", [(1, 2), (3, 31), (5, 512), (9, 513), (700, 1024), (33, 1000), (2, 2056), (17, 4096),
                                    (3, 8191), (2, 8200), (5, 16384), (2500, 96)])
def test_sizes(rows, D, dtype):
    _check(rows, D, dtype, F32, True, seed=D)
    _check(rows, D, dtype, BF, False, seed=D + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [8, 3])
def test_row_strides(pad, dtype):
    _check(40, 256, dtype, F32, True, pad=pad)


@pytest.mark.gpu
def test_large_mean_and_constant_rows():
    _check(50, 768, F32, F32, True, shift=30.0)
    x = torch.full((4, 64), 3.0, device=DEV)
    y, st = efla.efla_norm_fwd(x, torch.ones(64, device=DEV), None, eps=1e-5)
    efla.efla_get_status()
    assert float(y.abs().max()) == 0.0 and float((st[:, 0] - 3).abs().max()) == 0.0
    assert_close("rstd", st[:, 1], torch.full((4,), 1e-5, dtype=torch.float64).rsqrt(), TOL)


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    x = torch.randn(70, 300, device=DEV)
    w, b = torch.rand(300, device=DEV), torch.rand(300, device=DEV)
    y, st = efla.efla_norm_fwd(x, w, b)
    z = x.clone()
    z[13, 7], z[20, 8] = float("nan"), float("inf")
    y2, _ = efla.efla_norm_fwd(z, w, b)
    efla.efla_get_status()
    keep = [i for i in range(70) if i not in (13, 20)]
    assert torch.equal(y[keep], y2[keep]) and bool(y2[13].isnan().all()) and not bool(y2[20].isfinite().any())


@pytest.mark.gpu
def test_three_dimensions_streams_and_empty():
    x = torch.randn(3, 5, 128, device=DEV).to(BF)
    w = torch.rand(128, device=DEV)
    y, st = efla.efla_norm_fwd(x, w)
    assert y.shape == x.shape and st.shape == (3, 5, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, st2 = efla.efla_norm_fwd(x, w, stream=side)
    g2 = efla.efla_norm_bwd(x, w, y2, st2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = efla.efla_norm_bwd(x, w, y, st)
    assert torch.equal(y, y2) and all(torch.equal(p, r) for p, r in zip(g, g2))
    e = torch.empty(0, 128, device=DEV)
    ye, se = efla.efla_norm_fwd(e, w)
    dx, dw, db = efla.efla_norm_bwd(e, w, e, se)
    efla.efla_get_status()
    assert ye.shape == e.shape and float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0


@pytest.mark.gpu
def test_gradient_against_differences():
    """(f(x + h u) - f(x - h u)) / 2h of the GPU forward (fp32, D = 64) against <dx, u>: h = 1e-2 leaves
    truncation h^2 and rounding 1e-6 / h, each about 1e-4 of the scale."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, u, dy = (torch.randn(16, 64, generator=gen, device=DEV) for _ in range(3))
    w = torch.rand(64, generator=gen, device=DEV)
    _, st = efla.efla_norm_fwd(x, w)
    dx, _, _ = efla.efla_norm_bwd(x, w, dy, st)
    f = [float((efla.efla_norm_fwd(x + s * 1e-2 * u, w)[0].double() * dy.double()).sum()) for s in (1, -1)]
    want = float((dx.double() * u.double()).sum())
    assert abs((f[0] - f[1]) / 2e-2 - want) <= 1e-2 * max(abs(want), float(dx.norm()))


def test_refusals():
    """Host checks: nothing is launched (no GPU needed)."""
    import ctypes
    lib = efla.load_library()
    A = 0x7f0000000000
    p = [A + i * 0x10000000 for i in range(8)]

    def fwd(x=p[0], w=p[1], b=None, y=p[2], st=p[3], **kw):
        s = dict(rows=4, D=64, x_stride=64, y_stride=64, dtype=efla.BF16, weight_dtype=efla.F32, eps=1e-5)
        s.update(kw)
        return lib.efla_norm_fwd(ctypes.byref(efla.NormShape(**s)), x, w, b, y, st, None)

    def bwd(ws=p[7], n=1 << 30, dx=p[4], dw=p[5], db=p[6], **kw):
        s = dict(rows=4, D=64, x_stride=64, y_stride=64, dtype=efla.BF16, weight_dtype=efla.F32, eps=1e-5)
        s.update(kw)
        return lib.efla_norm_bwd(ctypes.byref(efla.NormShape(**s)), p[0], p[1], p[2], p[3], dx, dw, db, ws, n, None)

    assert lib.efla_norm_fwd(None, *p[:5], None) == 1
    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(st=None) == 1 and fwd(w=None) == 1
    assert fwd(rows=-1) == 1 and fwd(D=0) == 2 and fwd(D=16385) == 2 and fwd(dtype=9) == 2 and fwd(weight_dtype=9) == 2
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(x_stride=63) == 1 and fwd(y_stride=0) == 1
    assert fwd(x=p[0] + 1) == 3 and fwd(st=p[3] + 2) == 3
    assert fwd(y=p[0]) == 1 and fwd(st=p[1]) == 1
    assert fwd(rows=0, x=None) == 0
    assert bwd(ws=None) == 4 and bwd(n=16) == 4 and bwd(ws=p[7] + 4) == 3
    assert bwd(dx=p[2]) == 1 and bwd(dw=None) == 1 and bwd(db=p[5]) == 1
    assert lib.efla_last_error().decode()
