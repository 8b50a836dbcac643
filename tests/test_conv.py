"""The short causal convolution on the GPU against the 64-bit reference: max |err| / rms <= 1e-5.  A value is W + 1 products
and sums (2^-24 of each), then a sigmoid whose exponent is rounded to |x| 2^-24: under 2e-6 at the |x| <= 15 met here.  dw and
db add up to 1000 terms in runs of at most 64 (sqrt(64) 2^-24 of a run's rms at random, then eight and a few of those), and each
term is as exact as y: under 5e-6.  Values stored in bf16 add half an ulp."""
import ctypes

import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import mix
from parity import assert_close

TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def spans(B, L, lens):
    """Where the sequences lie on the axis of all tokens."""
    lens = [L] * B if lens is None else lens
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    return list(zip(ends, ends[1:]))


def make(B, L, D, W, dtype, wdtype=F32, bias=True, state=True, lens=None, pad=None, seed=0):
    """Tensors on the CPU; x as a slice of rows `pad` columns wider."""
    g = torch.Generator().manual_seed(seed + 1000 * D + L)
    seqs = spans(B, L, lens)
    T, n = seqs[-1][1] if seqs else 0, len(seqs)

    def rnd(*s):
        return torch.randn(*s, generator=g)

    return dict(seqs=seqs, x=rnd(T, D).to(dtype), w=(rnd(D, W) / 2).to(wdtype), b=(0.2 * rnd(D)).to(wdtype) if bias else None,
                S0=rnd(n, W - 1, D).to(dtype) if state else None, dy=rnd(T, D).to(dtype),
                dS=rnd(n, W - 1, D).to(dtype) if state else None, pad=pad, packed=lens is not None, B=B, L=L)


def gpu(t, name="x", a=None):
    """On the GPU; token arrays as slices of wider rows where the case says so, and in [B,L,D] unless packed."""
    if t is None:
        return None
    if a is None:
        return t.to(DEV)
    t = t if a["packed"] else t.view(a["B"], a["L"], t.shape[-1])
    if a["pad"] is None:
        return t.to(DEV)
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + a["pad"],), float("nan"), dtype=t.dtype, device=DEV)
    return wide[..., a["pad"]:].copy_(t)


def offsets(a):
    return torch.tensor([0] + [e for _, e in a["seqs"]], dtype=torch.int32, device=DEV) if a["packed"] else None


def d64(t):
    return None if t is None else t.double()


def check(silu=True, **kw):
    a = make(**kw)
    bf, wbf = a["x"].dtype == BF, a["w"].dtype == BF
    xs, dys = gpu(a["x"], "x", a), gpu(a["dy"], "dy", a)
    w, b, S0, dS = (gpu(a[n]) for n in ("w", "b", "S0", "dS"))
    off = offsets(a)
    y, last = efla.efla_conv_fwd(xs, w, b, S0, offsets=off, silu=silu)
    dx, dw, db, dS0 = efla.efla_conv_bwd(xs, w, dys, b, S0, dS, offsets=off, silu=silu, want_dS0=S0 is not None)
    efla.efla_get_status()
    args = [a["seqs"], d64(a["x"]), d64(a["w"]), d64(a["b"]), d64(a["S0"]), silu]
    y_ref, last_ref = mix.conv_all(*args)
    ref = mix.grads(lambda *t: mix.conv_all(a["seqs"], *t), args[1:], d64(a["dy"]), d64(a["dS"]))
    assert_close("y", y.flatten(0, -2), y_ref, TOL, stored_bf16=bf)
    assert torch.equal(last.cpu().double(), last_ref)
    assert_close("dx", dx.flatten(0, -2), ref[0], TOL, stored_bf16=bf)
    assert_close("dw", dw, ref[1], TOL, stored_bf16=wbf)
    if b is not None:
        assert_close("db", db, ref[2], TOL, stored_bf16=wbf)
    else:
        assert db is None
    if S0 is not None:
        assert_close("dS0", dS0, ref[3], TOL, stored_bf16=bf)
    again = efla.efla_conv_bwd(xs, w, dys, b, S0, dS, offsets=off, silu=silu, want_dS0=S0 is not None)
    assert all(p is q or torch.equal(p, q) for p, q in zip((dx, dw, db, dS0), again))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (2, 2, 1), (1, 3, 40), (2, 33, 64), (3, 70, 129), (1, 257, 1000)])
def test_sizes(B, L, D, W, dtype):
    check(B=B, L=L, D=D, W=W, dtype=dtype)
    check(B=B, L=L, D=D, W=W, dtype=dtype, wdtype=BF, bias=False, state=False, silu=False, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [8, 4, 3])
def test_slices_of_wider_rows(pad, dtype):
    check(B=2, L=50, D=96, W=4, dtype=dtype, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5, 0, 1, 2, 3, 64, 33, 0], [0, 0, 0], [1] * 40, [200, 1, 199]])
def test_packed(lens, dtype):
    check(B=0, L=0, D=72, W=4, dtype=dtype, lens=lens)
    check(B=0, L=0, D=37, W=3, dtype=dtype, lens=lens, state=False)


@pytest.mark.gpu
def test_gaps_and_bad_offsets_stay_inside():
    """Tokens outside every sequence keep what their outputs hold; offsets past the axis, or going back, are clamped."""
    a = make(B=1, L=40, D=16, W=4, dtype=F32)
    x, dy, w, b = gpu(a["x"]), gpu(a["dy"]), gpu(a["w"]), gpu(a["b"])
    off = torch.tensor([7, 20, 31], dtype=torch.int32, device=DEV)
    y = torch.full_like(x, 77.0)
    dx = torch.full_like(x, 77.0)
    efla.efla_conv_fwd(x, w, b, offsets=off, y=y)
    efla.efla_conv_bwd(x, w, dy, b, offsets=off, dx=dx)
    y_ref, _ = mix.conv_all([(7, 20), (20, 31)], d64(a["x"]), d64(a["w"]), d64(a["b"]), None, True)
    assert_close("y", y[7:31], y_ref, TOL)
    assert bool((y[:7] == 77).all()) and bool((y[31:] == 77).all()) and bool((dx[:7] == 77).all()) and bool((dx[31:] == 77).all())
    guard = torch.full((60, 16), 5.0, device=DEV)
    for bad in ([-5, 20, 4000], [30, 10, 20], [50, 60, 70]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        _, S = efla.efla_conv_fwd(x, w, b, offsets=off, y=guard[10:50])
        g = efla.efla_conv_bwd(x, w, dy, b, offsets=off, dx=guard[10:50])
        efla.efla_get_status()
        assert bool((guard[:10] == 5).all()) and bool((guard[50:] == 5).all()) and S.shape == (2, 3, 16) and g[1].shape == (16, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,W", [(64, 4), (37, 3), (8, 2)])
def test_tokens_one_by_one_are_the_sequence(D, W, dtype):
    """The step on a cache, in any order of places, gives the sequence's outputs and states, bit for bit."""
    B, L, n = 3, 6, 5
    a = make(B=B, L=L, D=D, W=W, dtype=dtype)
    x, w, b = gpu(a["x"], "x", a), gpu(a["w"]), gpu(a["b"])
    cache = torch.randn(n, W - 1, D, device=DEV).to(dtype)
    before = cache.clone()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    y, last = efla.efla_conv_fwd(x, w, b, cache[slots.long()])
    outs = [efla.efla_conv_step(x[:, t], w, cache, b, slots=slots) for t in range(L)]
    efla.efla_get_status()
    assert torch.equal(torch.stack(outs, 1), y) and torch.equal(cache[slots.long()], last)
    assert torch.equal(cache[[1, 3]], before[[1, 3]])


@pytest.mark.gpu
def test_step_skips_places_outside():
    x, w = torch.randn(4, 24, device=DEV), torch.randn(24, 4, device=DEV)
    cache = torch.randn(3, 3, 24, device=DEV)
    before = cache.clone()
    slots = torch.tensor([-1, 3, 1, 1 << 30], dtype=torch.int32, device=DEV)
    y = efla.efla_conv_step(x, w, cache, slots=slots)
    efla.efla_get_status()
    assert float(y[[0, 1, 3]].abs().max()) == 0.0 and torch.equal(cache[[0, 2]], before[[0, 2]])
    assert torch.equal(cache[1, :2], before[1, 1:]) and torch.equal(cache[1, 2], x[2])


@pytest.mark.gpu
def test_state_carries_a_cut_sequence():
    a = make(B=2, L=90, D=48, W=4, dtype=F32, state=False)
    x, w, b = gpu(a["x"], "x", a), gpu(a["w"]), gpu(a["b"])
    y, last = efla.efla_conv_fwd(x, w, b)
    y1, s1 = efla.efla_conv_fwd(x[:, :2], w, b)
    y2, s2 = efla.efla_conv_fwd(x[:, 2:], w, b, s1)
    efla.efla_get_status()
    assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(s2, last)


@pytest.mark.gpu
def test_no_tokens():
    w, b = torch.randn(16, 4, device=DEV), torch.randn(16, device=DEV)
    S0, dS = torch.randn(2, 3, 16, device=DEV), torch.randn(2, 3, 16, device=DEV)
    x = torch.empty(2, 0, 16, device=DEV)
    y, last = efla.efla_conv_fwd(x, w, b, S0)
    dx, dw, db, dS0 = efla.efla_conv_bwd(x, w, x, b, S0, dS)
    efla.efla_get_status()
    assert y.shape == x.shape and torch.equal(last, S0) and torch.equal(dS0, dS)
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0
    none = torch.empty(0, 5, 16, device=DEV)
    _, dw, db, _ = efla.efla_conv_bwd(none, w, none, b)
    assert float(dw.abs().max()) == 0.0 and float(db.abs().max()) == 0.0


@pytest.mark.gpu
def test_no_sequences():
    """offsets of one entry: nothing lies in a sequence."""
    x, w = torch.randn(5, 16, device=DEV), torch.randn(16, 4, device=DEV)
    off = torch.zeros(1, dtype=torch.int32, device=DEV)
    y, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    _, S = efla.efla_conv_fwd(x, w, offsets=off, y=y)
    _, dw, _, dS0 = efla.efla_conv_bwd(x, w, x, offsets=off, dx=dx)
    efla.efla_get_status()
    assert S.shape == dS0.shape == (0, 3, 16) and bool((y == 7).all()) and bool((dx == 7).all()) and float(dw.abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 37])
def test_gradient_into_a_slice(D):
    a = make(B=2, L=50, D=D, W=4, dtype=BF)
    x, dy, w = gpu(a["x"], "x", a), gpu(a["dy"], "dy", a), gpu(a["w"])
    want = efla.efla_conv_bwd(x, w, dy)
    rows = torch.full((2, 50, 2 * D + 8), 9.0, dtype=BF, device=DEV)
    got = efla.efla_conv_bwd(x, w, dy, dx=rows[..., D:2 * D])
    efla.efla_get_status()
    assert torch.equal(rows[..., D:2 * D], want[0]) and torch.equal(got[1], want[1])
    assert bool((rows[..., :D] == 9).all()) and bool((rows[..., 2 * D:] == 9).all())


@pytest.mark.gpu
def test_gradient_against_differences():
    """(f(x + h v) - f(x - h v)) / 2h of the GPU forward (fp32) against <dx, v>: h = 1e-2 leaves truncation h^2 and rounding
    1e-6 / h, each about 1e-4 of the scale."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x, v, dy = (torch.randn(2, 30, 40, generator=g, device=DEV) for _ in range(3))
    w = torch.randn(40, 4, generator=g, device=DEV) / 2
    dx = efla.efla_conv_bwd(x, w, dy, want_dS0=False)[0]
    f = [float((efla.efla_conv_fwd(x + s * 1e-2 * v, w)[0].double() * dy.double()).sum()) for s in (1, -1)]
    want = float((dx.double() * v.double()).sum())
    assert abs((f[0] - f[1]) / 2e-2 - want) <= 1e-2 * max(abs(want), float(dx.norm()))


@pytest.mark.gpu
def test_streams_and_graphs():
    a = make(B=2, L=100, D=64, W=4, dtype=BF)
    x, dy, w, b, S0 = gpu(a["x"], "x", a), gpu(a["dy"], "dy", a), gpu(a["w"]), gpu(a["b"]), gpu(a["S0"])
    want = efla.efla_conv_fwd(x, w, b, S0) + efla.efla_conv_bwd(x, w, dy, b, S0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = efla.efla_conv_fwd(x, w, b, S0, stream=side) + efla.efla_conv_bwd(x, w, dy, b, S0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = efla.efla_conv_fwd(x, w, b, S0) + efla.efla_conv_bwd(x, w, dy, b, S0)
    x.copy_(torch.randn_like(x))
    want = efla.efla_conv_fwd(x, w, b, S0) + efla.efla_conv_bwd(x, w, dy, b, S0)
    graph.replay()
    efla.efla_get_status()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


A = 0x7f0000000000
P = [A + i * 0x40000000 for i in range(14)]


def shape(**kw):
    s = dict(B=2, L=100, D=64, W=4, dtype=efla.BF16, weight_dtype=efla.F32, silu=1, packed=0)
    st = {n + "_stride": kw.pop(n + "_s", (6400, 64)) for n in ("x", "y", "dy", "dx")}
    s.update(kw)
    c = efla.ConvShape(**s)
    for n, v in st.items():
        setattr(c, n, type(getattr(c, n))(*v))
    return c


def test_refusals_forward():
    """Host checks: nothing is launched (no GPU needed)."""
    lib = efla.load_library()

    def fwd(off=None, x=P[0], w=P[1], b=P[2], S0=P[3], y=P[4], Sf=P[5], **kw):
        return lib.efla_conv_fwd(ctypes.byref(shape(**kw)), off, x, w, b, S0, y, Sf, None)

    assert lib.efla_conv_fwd(None, None, *P[:6], None) == 1
    for n in ("x", "w", "y"):
        assert fwd(**{n: None}) == 1, n
    assert fwd(B=-1) == 1 and fwd(L=-1) == 1 and fwd(packed=2) == 1 and fwd(silu=3) == 1
    assert fwd(D=0) == 2 and fwd(D=70000) == 2 and fwd(W=1) == 2 and fwd(W=5) == 2 and fwd(dtype=9) == 2 and fwd(weight_dtype=9) == 2
    assert fwd(L=(1 << 30) + 1) == 2 and fwd(B=1 << 20, L=1 << 20) == 2
    assert fwd(x=P[0] + 1) == 3 and fwd(w=P[1] + 2) == 3 and fwd(S0=P[3] + 1) == 3 and fwd(Sf=P[5] + 1) == 3
    assert fwd(y=P[0]) == 1 and fwd(Sf=P[3]) == 1 and fwd(Sf=P[0]) == 1 and fwd(y=P[1]) == 1 and fwd(Sf=P[4]) == 1
    assert fwd(x_s=(-1, 64)) == 1
    assert fwd(y_s=(6400, 32)) == 1 and b"y" in lib.efla_last_error()      # rows overlap
    assert fwd(packed=1) == 1 and fwd(packed=1, off=P[8] + 2) == 3 and fwd(packed=1, off=P[4]) == 1
    assert fwd(B=0, x=None, y=None) == 0


def test_refusals_backward_and_step():
    lib = efla.load_library()

    def bwd(off=None, x=P[0], w=P[1], b=P[2], S0=P[3], dy=P[4], dS=P[5], dx=P[6], dw=P[7], db=P[8], dS0=P[9], ws=P[10], n=1 << 29, **kw):
        return lib.efla_conv_bwd(ctypes.byref(shape(**kw)), off, x, w, b, S0, dy, dS, dx, dw, db, dS0, ws, n, None)

    for n in ("x", "w", "dy", "dx", "dw"):
        assert bwd(**{n: None}) == 1, n
    assert bwd(b=None) == 1 and bwd(dx=P[0]) == 1 and bwd(dw=P[1]) == 1 and bwd(dS0=P[5]) == 1 and bwd(db=P[7]) == 1 and bwd(ws=P[6]) == 1
    assert bwd(ws=None) == 4 and bwd(n=16) == 4 and bwd(ws=P[10] + 4) == 3
    # dx beside x in one buffer's token rows is apart from it; shifted by one element it is not
    # (a refused workspace proves that the aliasing check passed: it comes first)
    st = dict(x_s=(12800, 128), dx_s=(12800, 128))
    assert lib.efla_conv_bwd(ctypes.byref(shape(**st)), None, P[0], *P[1:6], P[0] + 128, *P[7:10], None, 0, None) == 4
    assert lib.efla_conv_bwd(ctypes.byref(shape(**st)), None, P[0], *P[1:6], P[0] + 126, *P[7:10], None, 0, None) == 1

    def step(x=P[0], w=P[1], b=P[2], S=P[3], slots=None, n=2, y=P[4], **kw):
        return lib.efla_conv_step(ctypes.byref(shape(**dict(dict(L=1), **kw))), x, w, b, S, slots, n, y, None)

    assert step(L=2) == 1 and step(packed=1) == 1 and step(S=None) == 1 and step(n=1) == 1 and step(n=-1) == 1 and step(x=None) == 1
    assert step(y=P[3]) == 1 and step(S=P[0]) == 1 and step(slots=P[5] + 1) == 3 and step(slots=P[3]) == 1 and step(y=P[0]) == 1
    assert step(B=0, n=0, S=None, x=None, y=None) == 0
    assert lib.efla_conv_bwd_workspace_size(ctypes.byref(shape())) > 0
    assert lib.efla_conv_bwd_workspace_size(ctypes.byref(shape(W=9))) == 0
