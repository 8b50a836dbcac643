"""The residual's RMS norm on the GPU against the 64-bit reference: max |err| / rms <= 1e-5 (sums of up to 16384 fp32 terms in
trees, about log2(D) 2^-24 each, and 2^-24 a multiply; dweight adds rows / CTAs terms one after another, sqrt(rows) 2^-24 at
most).  Values stored in bf16 add half an ulp; in e4m3 half a step: 2^-4 of the value, or 2^-10 of the scale below 2^-6."""
import ctypes

import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import mix
from parity import assert_close

TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def rows_of(rows, D, pad, dtype, gen, scale=1.0):
    t = (scale * torch.randn(rows, D, generator=gen)).to(dtype)
    return t, torch.empty(rows, D + pad, dtype=dtype, device=DEV)[:, :D].copy_(t)


def check(rows, D, dtype, wdtype=F32, residual=True, pad=0, eps=1e-5, seed=0):
    gen = torch.Generator().manual_seed(seed + D)
    x, xg = rows_of(rows, D, pad, dtype, gen)
    res, rg = rows_of(rows, D, pad, dtype, gen, 2.0)
    dy, dyg = rows_of(rows, D, pad, dtype, gen)
    dh, dhg = rows_of(rows, D, pad, dtype, gen)
    w = (1 + 0.2 * torch.randn(D, generator=gen)).to(wdtype)
    bf = dtype == BF
    if not residual:
        res = rg = dh = dhg = None
    y, scale, h, rstd = efla.efla_rms_fwd(xg, w.to(DEV), rg, eps=eps)
    want_h = x if res is None else (x.float() + res.float()).to(dtype)
    assert torch.equal(h.cpu(), want_h) and scale is None
    y_ref, r_ref = mix.rms_fwd(want_h.double(), w.double(), eps)
    assert_close("y", y, y_ref, TOL, stored_bf16=bf)
    assert_close("rstd", rstd, r_ref, TOL)
    dx, dw = efla.efla_rms_bwd(h, w.to(DEV), dyg, rstd, dh=dhg)
    efla.efla_get_status()
    ref = mix.rms_bwd(want_h.double(), w.double(), dy.double(), eps, None if dh is None else dh.double())
    # dx is a difference of terms of the size of rstd w dy: where it cancels (D = 1, where it is eps / h^2 of them) they are its scale
    terms = float((r_ref[:, None] * w.double() * dy.double()).square().mean().sqrt())
    lift = max(1.0, terms / float(ref[0].square().mean().sqrt())) if D <= 2 else 1.0
    assert_close("dx", dx, ref[0], lift * TOL, stored_bf16=bf)
    assert_close("dw", dw, ref[1], 2 * TOL, stored_bf16=wdtype == BF)
    again = efla.efla_rms_bwd(h, w.to(DEV), dyg, rstd, dh=dhg)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw), again))
    for group in {128, D}:
        q, scale, h8, r8 = efla.efla_rms_fwd(xg, w.to(DEV), rg, eps=eps, group=group)
        efla.efla_get_status()
        assert torch.equal(h8.cpu(), want_h) and torch.equal(r8, rstd)
        n = -(-D // group)
        assert scale.shape == (rows, n) and q.dtype == torch.float8_e4m3fn
        tops = torch.nn.functional.pad(y_ref.abs(), (0, n * group - D)).view(rows, n, group).amax(-1)
        assert_close("scale", scale, tops / 448, TOL)
        s = scale.cpu().double().repeat_interleave(group, 1)[:, :D]
        err = (q.cpu().double() * s - y_ref).abs()
        step = torch.maximum(y_ref.abs() * 2.0 ** -4, s * 2.0 ** -10)
        assert bool((err <= step * (1 + 1e-3) + TOL * y_ref.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 31), (5, 128), (4, 129), (5, 512), (9, 513), (700, 1024), (33, 1000), (2, 2056), (17, 4096),
                                    (3, 8191), (2, 8200), (5, 16384), (2500, 96)])
def test_sizes(rows, D, dtype):
    check(rows, D, dtype)
    check(rows, D, dtype, BF, residual=False, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [8, 3])
def test_row_strides(pad, dtype):
    check(40, 256, dtype, pad=pad)
    check(40, 1160, dtype, residual=False, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,D", [(40000, 64), (20000, 1024), (4500, 4096), (1600, 8192), (1500, 16384), (5000, 333)])
def test_many_rows_a_group(rows, D, dtype):
    """Every group of warps takes ten rows and more: the ring's stages are filled again and change phase."""
    check(rows, D, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [256, 1000, 4096])
def test_in_place(D):
    """h over x or over the residual, dx over dh: the same values as apart."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r, dy, dh = (torch.randn(300, D, generator=g, device=DEV).to(BF) for _ in range(4))
    w = torch.rand(D, generator=g, device=DEV)
    want = efla.efla_rms_fwd(x, w, r)
    for target in ("x", "r"):
        a, b = x.clone(), r.clone()
        got = efla.efla_rms_fwd(a, w, b, h=a if target == "x" else b)
        assert all(p is q or torch.equal(p, q) for p, q in zip(got, want))
    dx, dw = efla.efla_rms_bwd(want[2], w, dy, want[3], dh=dh)
    dx2, dw2 = efla.efla_rms_bwd(want[2], w, dy, want[3], dh=dh, dx=dh)
    efla.efla_get_status()
    assert dx2 is dh and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [512, 515])
def test_zero_rows_and_extremes_in_8_bits(D):
    x = torch.randn(6, D, device=DEV)
    x[1] = 0
    x[2, 1:] = 0                       # one value: scale its own
    x[3] *= 1e-30
    x[4] *= 1e15
    w = torch.ones(D, device=DEV)
    for group in (128, D):
        q, scale, _, _ = efla.efla_rms_fwd(x, w, eps=1e-5, group=group)
        efla.efla_get_status()
        v = q.float() * scale.repeat_interleave(group, 1)[:, :D]
        assert bool(torch.isfinite(v).all()) and float(v[1].abs().max()) == 0.0 and float(scale[1].max()) == 2.0 ** -126
        y = efla.efla_rms_fwd(x, w, eps=1e-5)[0]
        assert bool(((v - y).abs() <= torch.maximum(y.abs() / 15.9, scale.repeat_interleave(group, 1)[:, :D] / 1000)).all())
        assert float(q.float().abs().max()) == 448.0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [300, 304])
def test_nan_stays_in_its_row(D):
    x, r = torch.randn(70, D, device=DEV), torch.randn(70, D, device=DEV)
    w = torch.rand(D, device=DEV)
    y, _, h, _ = efla.efla_rms_fwd(x, w, r)
    q, s, _, _ = efla.efla_rms_fwd(x, w, r, group=128)
    z = x.clone()
    z[13, 7], z[20, 8] = float("nan"), float("inf")
    y2, _, h2, _ = efla.efla_rms_fwd(z, w, r)
    q2, s2, _, _ = efla.efla_rms_fwd(z, w, r, group=128)
    efla.efla_get_status()
    keep = [i for i in range(70) if i not in (13, 20)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(h[keep], h2[keep]) and bool(y2[13].isnan().all()) and bool(y2[20, 8].isnan())
    assert torch.equal(q[keep].view(torch.uint8), q2[keep].view(torch.uint8)) and torch.equal(s[keep], s2[keep])
    assert bool(q2[13].float().isnan().all())


@pytest.mark.gpu
def test_three_dimensions_streams_graphs_and_empty():
    x, r = torch.randn(3, 5, 128, device=DEV).to(BF), torch.randn(3, 5, 128, device=DEV).to(BF)
    w = torch.rand(128, device=DEV)

    def both(**kw):
        y, _, h, rstd = efla.efla_rms_fwd(x, w, r, **kw)
        q, s, _, _ = efla.efla_rms_fwd(x, w, r, group=128, **kw)
        return (y, h, rstd, q.view(torch.uint8), s) + efla.efla_rms_bwd(h, w, y, rstd, dh=r, **kw)

    want = both()
    assert want[0].shape == x.shape and want[2].shape == (3, 5) and want[4].shape == (3, 5, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    x.copy_(torch.randn_like(x))
    want = both()
    graph.replay()
    efla.efla_get_status()
    assert all(torch.equal(p, q) for p, q in zip(out, want))
    e = torch.empty(0, 128, device=DEV)
    y, s, h, rstd = efla.efla_rms_fwd(e, w, e.clone(), group=128)
    dx, dw = efla.efla_rms_bwd(e, w, e, rstd)
    efla.efla_get_status()
    assert y.shape == e.shape and s.shape == (0, 1) and dx.shape == e.shape and float(dw.abs().max()) == 0.0


@pytest.mark.gpu
def test_gradient_against_differences():
    """(f(x + h u) - f(x - h u)) / 2h of the GPU forward (fp32, D = 64) against <dx, u>: h = 1e-2 leaves
    truncation h^2 and rounding 1e-6 / h, each about 1e-4 of the scale."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, u, dy = (torch.randn(16, 64, generator=gen, device=DEV) for _ in range(3))
    w = torch.rand(64, generator=gen, device=DEV)
    rstd = efla.efla_rms_fwd(x, w)[3]
    dx, _ = efla.efla_rms_bwd(x, w, dy, rstd)
    f = [float((efla.efla_rms_fwd(x + s * 1e-2 * u, w)[0].double() * dy.double()).sum()) for s in (1, -1)]
    want = float((dx.double() * u.double()).sum())
    assert abs((f[0] - f[1]) / 2e-2 - want) <= 1e-2 * max(abs(want), float(dx.norm()))


def test_refusals():
    """Host checks: nothing is launched (no GPU needed)."""
    lib = efla.load_library()
    p = [0x7f0000000000 + i * 0x10000000 for i in range(10)]
    base = dict(rows=4, D=256, group=0, x_stride=256, residual_stride=256, y_stride=256, h_stride=256, dy_stride=256, dh_stride=256,
                dx_stride=256, dtype=efla.BF16, weight_dtype=efla.F32, eps=1e-5)

    def fwd(x=p[0], r=p[1], w=p[2], y=p[3], sc=p[4], h=p[5], rs=p[6], **kw):
        return lib.efla_rms_fwd(ctypes.byref(efla.RmsShape(**dict(base, **kw))), x, r, w, y, sc, h, rs, None)

    def bwd(h=p[0], w=p[1], dy=p[2], rs=p[3], dh=p[4], dx=p[5], dw=p[6], ws=p[7], n=1 << 27, **kw):
        return lib.efla_rms_bwd(ctypes.byref(efla.RmsShape(**dict(base, **kw))), h, w, dy, rs, dh, dx, dw, ws, n, None)

    assert lib.efla_rms_fwd(None, *p[:7], None) == 1
    for n in ("x", "w", "y", "rs", "h", "r"):
        assert fwd(**{n: None}) == 1, n
    assert fwd(group=128, sc=None) == 1
    assert fwd(rows=-1) == 1 and fwd(D=0) == 2 and fwd(D=16385) == 2 and fwd(dtype=9) == 2 and fwd(weight_dtype=9) == 2
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1 and fwd(group=64) == 2 and fwd(group=-1) == 2
    assert fwd(x_stride=255) == 1 and fwd(residual_stride=0) == 1 and fwd(y_stride=8) == 1 and fwd(h_stride=8) == 1
    assert fwd(x=p[0] + 1) == 3 and fwd(rs=p[6] + 2) == 3 and fwd(w=p[2] + 1) == 3 and fwd(group=128, sc=p[4] + 1) == 3
    assert fwd(y=p[0]) == 1 and fwd(rs=p[2]) == 1 and fwd(h=p[3]) == 1 and fwd(h=p[2]) == 1
    assert fwd(h=p[0] + 16) == 1 and fwd(h=p[0], h_stride=264) == 1 and fwd(h=p[1], residual_stride=264) == 1
    assert fwd(rows=0, x=None, y=None, r=None, h=None) == 0
    for n in ("h", "w", "dy", "rs", "dx", "dw"):
        assert bwd(**{n: None}) == 1, n
    assert bwd(ws=None) == 4 and bwd(n=16) == 4 and bwd(ws=p[7] + 4) == 3
    assert bwd(dx=p[2]) == 1 and bwd(dw=p[1]) == 1 and bwd(dx=p[0]) == 1 and bwd(dw=p[4]) == 1 and bwd(dx=p[4] + 16) == 1
    assert bwd(dx=p[4], dx_stride=264) == 1
    assert bwd(dx=p[4], ws=None) == 4      # accepted up to its workspace: in place
    assert lib.efla_last_error().decode()
