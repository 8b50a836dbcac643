"""The selective scan on the GPU against the 64-bit reference: max |err| / rms <= 2e-5 for fp32 values.  A decay is ex2.approx
(2^-22 of it at most, -2e-8 on average) of a product rounded to 2^-24, so that a state that remembers m tokens is off by
m 2e-8 + sqrt(m) 6e-8 of itself: 8e-6 at the m <= 300 met here; sums over up to 64 states, 1000 channels or 1000 tokens in fp32
add a few 2^-24 sqrt(terms) of their rms.  Gradients of A weigh each state by both: they get twice that.  Values stored in
bf16 add half an ulp."""
import ctypes

import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import mix
from parity import assert_close
from test_conv import BF, DEV, F32, d64, gpu, offsets, spans

TOL = 2e-5
NAMES = ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "dbias", "dS0")


def make(B, L, D, N, G=1, dtype=F32, gate=True, skip=True, bias=True, softplus=True, state=True, lens=None, pad=None, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * D + 1000 * N + L)
    seqs = spans(B, L, lens)
    T, n = seqs[-1][1] if seqs else 0, len(seqs)

    def rnd(*s):
        return torch.randn(*s, generator=g)

    size = torch.exp(-4.6 * torch.rand(D, generator=g) - 0.5)      # step sizes from 0.006 to 0.6
    delta = 0.5 * rnd(T, D)
    if not bias:
        delta = delta - 2
    elif softplus:
        bias = size + torch.log(-torch.expm1(-size))
    else:
        bias = size
    if not softplus:
        delta = 0.1 * delta.abs()
    return dict(seqs=seqs, u=rnd(T, D).to(dtype), delta=delta.to(dtype), A=-torch.exp(0.5 * rnd(D, N)), B_=rnd(T, G * N).to(dtype),
                C=rnd(T, G * N).to(dtype), D=rnd(D) if skip else None, z=rnd(T, D).to(dtype) if gate else None,
                bias=bias if torch.is_tensor(bias) else None, S0=rnd(n, D, N) if state else None, dy=rnd(T, D).to(dtype),
                dS=rnd(n, D, N) if state else None, pad=pad, packed=lens is not None, B=B, L=L, G=G, N=N, softplus=softplus)


def on_gpu(a):
    t = {k: gpu(a[k], k, a) for k in ("u", "delta", "z", "dy")}
    t.update({k: gpu(a[k]) for k in ("A", "D", "bias", "S0", "dS")})
    t.update({k: gpu(a[k], k, a).unflatten(-1, (a["G"], a["N"])) for k in ("B_", "C")})
    return t


def reference(a):
    """(y, S_final) and the gradients in NAMES' order, in 64 bits."""
    bc = [d64(a[k]).view(-1, a["G"], a["N"]) for k in ("B_", "C")]
    args = [d64(a["u"]), d64(a["delta"]), d64(a["A"]), *bc, d64(a["D"]), d64(a["z"]), d64(a["bias"]), d64(a["S0"])]
    fn = lambda *t: mix.scan_all(a["seqs"], *t, a["softplus"])  # noqa: E731
    return fn(*args), mix.grads(fn, args, d64(a["dy"]), d64(a["dS"]))


def check(tol=TOL, **kw):
    a = make(**kw)
    t, bf, off = on_gpu(a), a["u"].dtype == BF, offsets(a)
    ins = (t["u"], t["delta"], t["A"], t["B_"], t["C"])
    rest = (t["D"], t["z"], t["bias"], t["S0"])
    kws = dict(offsets=off, softplus=a["softplus"])
    y, last = efla.efla_scan_fwd(*ins, *rest, **kws)
    got = efla.efla_scan_bwd(*ins, t["dy"], *rest, t["dS"], want_dS0=t["S0"] is not None, **kws)
    efla.efla_get_status()
    (y_ref, last_ref), ref = reference(a)
    lead = -2 if y.dim() == 2 else -3
    assert_close("y", y.reshape(y_ref.shape), y_ref, tol, stored_bf16=bf)
    assert_close("S_final", last, last_ref, tol)
    # dB and dC of D/G channels, ddelta and dA of N states are sums of both signs: their terms set the scale of a few
    for name, p, r in zip(NAMES, got, ref):
        if r is None:
            assert p is None, name
            continue
        stored = bf and name in ("du", "ddelta", "dB", "dC", "dz")
        assert_close(name, p.reshape(r.shape), r, (2 if name in ("dA", "dbias") else 1) * tol, stored_bf16=stored)
    again = efla.efla_scan_bwd(*ins, t["dy"], *rest, t["dS"], want_dS0=t["S0"] is not None, **kws)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, again)) and lead


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 4, 5, 8, 13, 16, 24, 32, 64])
def test_states(N, dtype):
    check(B=2, L=37, D=24, N=N, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,D,N,G", [(1, 1, 1, 16, 1), (1, 2, 3, 3, 3), (3, 15, 130, 16, 1), (2, 16, 128, 16, 2), (1, 17, 520, 4, 1),
                                       (2, 63, 260, 8, 1), (1, 64, 36, 32, 3), (1, 65, 70, 64, 2), (1, 300, 200, 16, 4)])
def test_sizes(B, L, D, N, G, dtype):
    check(B=B, L=L, D=D, N=N, G=G, dtype=dtype)
    check(B=B, L=L, D=D, N=N, G=G, dtype=dtype, gate=False, skip=False, bias=False, state=False, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(softplus=False), dict(softplus=False, bias=False), dict(gate=False), dict(skip=False, state=False)])
def test_options(kw):
    check(B=2, L=70, D=40, N=16, dtype=F32, **kw)
    check(B=2, L=70, D=40, N=16, dtype=BF, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [8, 4, 3])
def test_slices_of_wider_rows(pad, dtype):
    check(B=2, L=50, D=96, N=16, G=2, dtype=dtype, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5, 0, 1, 2, 3, 64, 33, 0], [0, 0, 0], [1] * 70, [200, 1, 183], [64, 64, 64], [300]])
def test_packed(lens, dtype):
    check(B=0, L=0, D=40, N=16, dtype=dtype, lens=lens)
    check(B=0, L=0, D=37, N=8, dtype=dtype, lens=lens, state=False, gate=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_segments(dtype):
    """Few channels and many tokens: the forward cuts the tokens into segments (256 tokens and more), batched and packed."""
    check(B=1, L=700, D=16, N=16, dtype=dtype)
    check(B=2, L=515, D=40, N=8, dtype=dtype, state=False)
    check(B=0, L=0, D=24, N=16, dtype=dtype, lens=[130, 0, 260, 1, 129, 380])
    shape = efla.ScanShape(B=1, L=700, D=16, G=1, N=16, dtype=efla.F32, softplus=1)
    assert efla.efla_scan_fwd_workspace_size(shape) > 0


@pytest.mark.gpu
def test_gaps_and_bad_offsets_stay_inside():
    """Tokens outside every sequence keep what their outputs hold; offsets past the axis, or going back, are clamped."""
    a = make(B=1, L=300, D=16, N=8, state=False)
    t = on_gpu(dict(a, packed=True))
    ins, rest = (t["u"], t["delta"], t["A"], t["B_"], t["C"]), (t["D"], t["z"], t["bias"])
    off = torch.tensor([7, 90, 271], dtype=torch.int32, device=DEV)
    y, du, dd, dz = (torch.full_like(t["u"], 77.0) for _ in range(4))
    # (what lies outside may be anything)
    for k in ("u", "delta", "z", "B_", "C", "dy"):
        t[k][:7] = float("nan")
        t[k][271:] = float("inf")
    _, last = efla.efla_scan_fwd(*ins, *rest, offsets=off, y=y)
    g = efla.efla_scan_bwd(*ins, t["dy"], *rest, offsets=off, du=du, ddelta=dd, dz=dz)
    efla.efla_get_status()
    inner = {k: a[k][7:271] for k in ("u", "delta", "z", "B_", "C", "dy")}
    (y_ref, last_ref), ref = reference(dict(a, seqs=[(0, 83), (83, 264)], **inner))
    assert_close("y", y[7:271], y_ref, TOL)
    assert_close("S_final", last, last_ref, TOL)
    assert_close("dA", g[2], ref[2], 2 * TOL)
    assert_close("dB", g[3][7:271], ref[3], TOL)
    for name, o, r in (("du", du, ref[0]), ("ddelta", dd, ref[1]), ("dz", dz, ref[6])):
        assert_close(name, o[7:271], r, TOL)
    for o in (y, du, dd, dz):
        assert bool((o[:7] == 77).all()) and bool((o[271:] == 77).all())
    guard = torch.full((340, 16), 5.0, device=DEV)
    for bad in ([-5, 20, 4000], [200, 10, 20], [400, 500, 600]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        efla.efla_scan_fwd(*ins, *rest, offsets=off, y=guard[20:320])
        efla.efla_scan_bwd(*ins, t["dy"], *rest, offsets=off, du=guard[20:320])
        efla.efla_get_status()
        assert bool((guard[:20] == 5).all()) and bool((guard[320:] == 5).all())


@pytest.mark.gpu
def test_masked_tokens_leave_the_state():
    """dt = 0 (delta far below zero) drops a token: e^0 h + 0, in every state and bit."""
    a = make(B=1, L=40, D=32, N=16, gate=False)
    t = on_gpu(a)
    t["delta"][:, 20:] = -200.0
    ins = (t["u"], t["delta"], t["A"], t["B_"], t["C"])
    _, whole = efla.efla_scan_fwd(*ins, t["D"], None, t["bias"], t["S0"])
    _, cut = efla.efla_scan_fwd(*(x[:, :20] if x.dim() > 2 else x for x in ins), t["D"], None, t["bias"], t["S0"])
    efla.efla_get_status()
    assert torch.equal(whole, cut)


@pytest.mark.gpu
def test_nan_stays_in_its_channel_and_sequence():
    a = make(B=0, L=0, D=40, N=16, lens=[40, 50, 30], dtype=F32, gate=False)
    t, off = on_gpu(a), offsets(a)
    ins, rest = [t["u"], t["delta"], t["A"], t["B_"], t["C"]], (t["D"], None, t["bias"], t["S0"])
    y, last = efla.efla_scan_fwd(*ins, *rest, offsets=off)
    u = t["u"].clone()
    u[60, 7] = float("nan")
    y2, last2 = efla.efla_scan_fwd(u, *ins[1:], *rest, offsets=off)
    efla.efla_get_status()
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[60:90, 7] = True
    assert torch.equal(y[~hit], y2[~hit]) and bool(y2[hit].isnan().all())
    assert bool(last2[1, 7].isnan().all())
    last2[1, 7] = last[1, 7]
    assert torch.equal(last, last2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,N,G", [(64, 16, 1), (37, 13, 1), (24, 64, 2), (6, 3, 3)])
def test_tokens_one_by_one_are_the_sequence(D, N, G, dtype):
    """The step on a cache, in any order of places, against the sequence's outputs and states."""
    B, L, n = 3, 6, 5
    a = make(B=B, L=L, D=D, N=N, G=G, dtype=dtype)
    t = on_gpu(a)
    cache = torch.randn(n, D, N, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    cache[slots.long()] = t["S0"]
    before = cache.clone()
    (y_ref, last_ref), _ = reference(a)
    outs = [efla.efla_scan_step(t["u"][:, i], t["delta"][:, i], t["A"], t["B_"][:, i], t["C"][:, i], cache, t["D"], t["z"][:, i],
                                t["bias"], slots=slots) for i in range(L)]
    efla.efla_get_status()
    assert_close("y", torch.stack(outs, 1).reshape(y_ref.shape), y_ref, TOL, stored_bf16=dtype == BF)
    assert_close("S", cache[slots.long()], last_ref, TOL)
    assert torch.equal(cache[[1, 3]], before[[1, 3]])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,D,N,G", [(255, 1200, 16, 1), (129, 1337, 13, 7), (301, 512, 64, 2), (700, 512, 8, 1), (1300, 96, 4, 3)])
def test_step_of_a_batch(B, D, N, G, dtype):
    """Batches that give a CTA several sequences, some CTAs fewer; odd widths."""
    a = make(B=B, L=1, D=D, N=N, G=G, dtype=dtype)
    t = on_gpu(a)
    cache = torch.randn(B + 3, D, N, device=DEV)
    slots = torch.randperm(B + 3, device=DEV)[:B].int()
    slots[5] = -1
    before = cache.clone()
    one = [t[k][:, 0] for k in ("u", "delta")]
    y = efla.efla_scan_step(*one, t["A"], t["B_"][:, 0], t["C"][:, 0], cache, t["D"], t["z"][:, 0], t["bias"], slots=slots)
    efla.efla_get_status()
    S, keep = before[slots.long().clamp_min(0)], torch.arange(B, device=DEV) != 5
    u, z, raw = t["u"][:, 0].double(), t["z"][:, 0].double(), t["delta"][:, 0].double() + t["bias"].double()
    dt = torch.nn.functional.softplus(raw, threshold=50)
    rep = D // G
    bm, c = (t[k][:, 0].double().repeat_interleave(rep, 1) for k in ("B_", "C"))
    h = torch.exp(dt[..., None] * t["A"].double()) * S.double() + (dt * u)[..., None] * bm
    want = ((h * c).sum(-1) + t["D"].double() * u) * z * torch.sigmoid(z)
    assert_close("y", y[keep], want[keep], TOL, stored_bf16=dtype == BF)
    assert float(y[5].abs().max()) == 0.0
    assert_close("S", cache[slots[keep].long()], h[keep], TOL)
    rest = torch.ones(B + 3, dtype=torch.bool, device=DEV)
    rest[slots[keep].long()] = False
    assert torch.equal(cache[rest], before[rest])


@pytest.mark.gpu
def test_step_skips_places_outside():
    a = make(B=4, L=1, D=24, N=16, state=False)
    t = on_gpu(a)
    cache = torch.randn(3, 24, 16, device=DEV)
    before = cache.clone()
    slots = torch.tensor([-1, 3, 1, 1 << 30], dtype=torch.int32, device=DEV)
    y = efla.efla_scan_step(*(t[k][:, 0] for k in ("u", "delta")), t["A"], t["B_"][:, 0], t["C"][:, 0], cache, t["D"], slots=slots)
    efla.efla_get_status()
    assert float(y[[0, 1, 3]].abs().max()) == 0.0 and torch.equal(cache[[0, 2]], before[[0, 2]]) and not torch.equal(cache[1], before[1])


@pytest.mark.gpu
def test_state_carries_a_cut_sequence():
    a = make(B=2, L=90, D=48, N=16, state=False)
    t = on_gpu(a)
    cut = lambda x, i: x if x is None or x.dim() < 3 else (x[:, :33], x[:, 33:])[i]  # noqa: E731
    args = [t[k] for k in ("u", "delta", "A", "B_", "C", "D", "z", "bias")]
    y, last = efla.efla_scan_fwd(*args)
    y1, s1 = efla.efla_scan_fwd(*(cut(x, 0) for x in args))
    y2, s2 = efla.efla_scan_fwd(*(cut(x, 1) for x in args), s1)
    efla.efla_get_status()
    assert_close("y", torch.cat([y1, y2], 1), y.double().cpu(), TOL)
    assert_close("S", s2, last.double().cpu(), TOL)


@pytest.mark.gpu
def test_no_tokens():
    S0, dS = torch.randn(2, 16, 8, device=DEV), torch.randn(2, 16, 8, device=DEV)
    u, bc = torch.empty(2, 0, 16, device=DEV), torch.empty(2, 0, 1, 8, device=DEV)
    A, D = -torch.rand(16, 8, device=DEV), torch.rand(16, device=DEV)
    y, last = efla.efla_scan_fwd(u, u, A, bc, bc, D, None, D, S0)
    g = efla.efla_scan_bwd(u, u, A, bc, bc, u, D, None, D, S0, dS)
    efla.efla_get_status()
    assert y.shape == u.shape and torch.equal(last, S0) and torch.equal(g[8], dS)
    assert all(float(g[i].abs().max()) == 0.0 for i in (2, 5, 7))
    none, bn = torch.empty(0, 5, 16, device=DEV), torch.empty(0, 5, 1, 8, device=DEV)
    g = efla.efla_scan_bwd(none, none, A, bn, bn, none, D, None, D)
    efla.efla_get_status()
    assert all(float(g[i].abs().max()) == 0.0 for i in (2, 5, 7))


@pytest.mark.gpu
def test_no_sequences():
    """offsets of one entry: nothing lies in a sequence."""
    a = make(B=1, L=40, D=16, N=8, state=False)
    t = on_gpu(dict(a, packed=True))
    ins, rest = (t["u"], t["delta"], t["A"], t["B_"], t["C"]), (t["D"], t["z"], t["bias"])
    off = torch.zeros(1, dtype=torch.int32, device=DEV)
    y, du = torch.full_like(t["u"], 7.0), torch.full_like(t["u"], 7.0)
    _, S = efla.efla_scan_fwd(*ins, *rest, offsets=off, y=y)
    g = efla.efla_scan_bwd(*ins, t["dy"], *rest, offsets=off, du=du)
    efla.efla_get_status()
    assert S.shape == g[8].shape == (0, 16, 8) and bool((y == 7).all()) and bool((du == 7).all())
    assert all(float(g[i].abs().max()) == 0.0 for i in (2, 5, 7))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 37])
def test_gradients_into_slices_of_one_buffer(D, dtype):
    a = make(B=2, L=70, D=D, N=16, dtype=dtype)
    t = on_gpu(a)
    ins, rest = (t["u"], t["delta"], t["A"], t["B_"], t["C"]), (t["D"], t["z"], t["bias"], t["S0"], t["dS"])
    want = efla.efla_scan_bwd(*ins, t["dy"], *rest)
    rows = torch.full((2, 70, 3 * D + 4), 9.0, dtype=dtype, device=DEV)
    got = efla.efla_scan_bwd(*ins, t["dy"], *rest, du=rows[..., :D], ddelta=rows[..., D:2 * D], dz=rows[..., 2 * D:3 * D])
    efla.efla_get_status()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    assert bool((rows[..., 3 * D:] == 9).all())


@pytest.mark.gpu
def test_broadcast_inputs():
    """B and C of one row for a whole batch, and a gate of one row for every token: strides of zero."""
    a = make(B=3, L=33, D=32, N=16)
    t = on_gpu(a)
    b, c, z = t["B_"][:1].expand(3, -1, -1, -1), t["C"][:1].expand(3, -1, -1, -1), t["z"][:, :1].expand(-1, 33, -1)
    rest = (t["D"], t["bias"], t["S0"])
    for got, want in ((efla.efla_scan_fwd(t["u"], t["delta"], t["A"], b, c, rest[0], z, *rest[1:]),
                       efla.efla_scan_fwd(t["u"], t["delta"], t["A"], b.contiguous(), c.contiguous(), rest[0], z.contiguous(), *rest[1:])),
                      (efla.efla_scan_bwd(t["u"], t["delta"], t["A"], b, c, t["dy"], rest[0], z, *rest[1:]),
                       efla.efla_scan_bwd(t["u"], t["delta"], t["A"], b.contiguous(), c.contiguous(), t["dy"], rest[0], z.contiguous(), *rest[1:]))):
        efla.efla_get_status()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.gpu
def test_gradients_against_differences():
    """(f(x + h v) - f(x - h v)) / 2h of the GPU forward (fp32) against <dx, v>: h = 1e-2 leaves truncation h^2 and rounding
    1e-6 / h, each about 1e-4 of the scale."""
    a = make(B=1, L=40, D=24, N=8, state=False, bias=False)
    t = on_gpu(a)
    args = [t["u"], t["delta"], t["A"], t["B_"], t["C"], t["D"], t["z"]]
    g = efla.efla_scan_bwd(*args[:5], t["dy"], *args[5:], want_dS0=False)
    for i, name in enumerate(NAMES[:7]):
        v = torch.randn_like(args[i])
        f = [float((efla.efla_scan_fwd(*(x + s * 1e-2 * v if j == i else x for j, x in enumerate(args)))[0].double() * t["dy"].double()).sum())
             for s in (1, -1)]
        want = float((g[i].double() * v.double()).sum())
        assert abs((f[0] - f[1]) / 2e-2 - want) <= 1e-2 * max(abs(want), float(g[i].norm())), name


@pytest.mark.gpu
@pytest.mark.parametrize("L", [100, 600])
def test_streams_and_graphs(L):
    a = make(B=1, L=L, D=64, N=16, dtype=BF)
    t = on_gpu(a)
    ins, rest = (t["u"], t["delta"], t["A"], t["B_"], t["C"]), (t["D"], t["z"], t["bias"], t["S0"])

    def both(**kw):
        return efla.efla_scan_fwd(*ins, *rest, **kw) + efla.efla_scan_bwd(*ins, t["dy"], *rest, t["dS"], **kw)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    t["u"].copy_(torch.randn_like(t["u"]))
    want = both()
    graph.replay()
    efla.efla_get_status()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


P = [0x7f0000000000 + i * 0x40000000 for i in range(26)]


def shape(**kw):
    s = dict(B=2, L=100, D=64, G=2, N=16, dtype=efla.BF16, softplus=1, packed=0)
    st = {n + "_stride": kw.pop(n + "_s", (6400, 64)) for n in ("u", "delta", "z", "y", "dy", "du", "ddelta", "dz")}
    st.update({n + "_stride": kw.pop(n + "_s", (3200, 32, 16)) for n in ("B", "C")})
    s.update(kw)
    c = efla.ScanShape(**s)
    for n, v in st.items():
        setattr(c, n, type(getattr(c, n))(*v))
    return c


def test_refusals_forward_and_step():
    """Host checks: nothing is launched (no GPU needed)."""
    lib = efla.load_library()

    def fwd(off=None, u=P[0], dl=P[1], A=P[2], Bm=P[3], C=P[4], sk=P[5], z=P[6], bi=P[7], S0=P[8], y=P[9], Sf=P[10], ws=P[11], n=1 << 29, **kw):
        return lib.efla_scan_fwd(ctypes.byref(shape(**kw)), off, u, dl, A, Bm, C, sk, z, bi, S0, y, Sf, ws, n, None)

    assert lib.efla_scan_fwd(None, None, *P[:12], 1 << 29, None) == 1
    for n in ("u", "dl", "A", "Bm", "C", "y"):
        assert fwd(**{n: None}) == 1, n
    assert fwd(B=-1) == 1 and fwd(L=-1) == 1 and fwd(G=3) == 1 and fwd(G=0) == 1 and fwd(packed=2) == 1 and fwd(softplus=2) == 1
    assert fwd(N=0) == 2 and fwd(N=65) == 2 and fwd(D=0) == 2 and fwd(D=65538) == 2 and fwd(dtype=9) == 2 and fwd(L=(1 << 30) + 1) == 2
    assert fwd(B=65536) == 2 and fwd(B=60000, L=1 << 28) == 2
    assert fwd(u=P[0] + 1) == 3 and fwd(S0=P[8] + 4) == 3 and fwd(A=P[2] + 2) == 3 and fwd(Sf=P[10] + 8) == 3 and fwd(ws=P[11] + 4) == 3
    assert fwd(y=P[0]) == 1 and fwd(y=P[6]) == 1 and fwd(Sf=P[8]) == 1 and fwd(Sf=P[2]) == 1 and fwd(y=P[3]) == 1 and fwd(Sf=P[9]) == 1
    assert fwd(u_s=(-1, 64)) == 1 and fwd(B_s=(3200, -1, 16)) == 1 and fwd(y_s=(6400, 60)) == 1
    assert fwd(packed=1) == 1 and fwd(packed=1, off=P[12] + 2) == 3 and fwd(packed=1, off=P[9]) == 1
    long = dict(L=1000, y_s=(64000, 64))     # (few channels, many tokens: segments)
    assert fwd(ws=None, **long) == 4 and fwd(n=64, **long) == 4
    assert fwd(B=0, u=None, y=None, ws=None) == 0

    def step(u=P[0], S=P[8], slots=None, n=2, y=P[9], **kw):
        return lib.efla_scan_step(ctypes.byref(shape(**dict(dict(L=1), **kw))), u, *P[1:8], S, slots, n, y, None)

    assert step(L=2) == 1 and step(packed=1) == 1 and step(S=None) == 1 and step(n=1) == 1 and step(n=-1) == 1 and step(u=None) == 1
    assert step(y=P[8]) == 1 and step(S=P[2]) == 1 and step(S=P[8] + 8) == 3 and step(slots=P[12] + 1) == 3 and step(slots=P[8]) == 1
    assert step(B=0, n=0, S=None, u=None, y=None) == 0


def test_refusals_backward():
    lib = efla.load_library()

    def bwd(off=None, u=P[0], dl=P[1], A=P[2], Bm=P[3], C=P[4], sk=P[5], z=P[6], bi=P[7], S0=P[8], dy=P[9], dS=P[10], du=P[11], dd=P[12],
            dA=P[13], dB=P[14], dC=P[15], dsk=P[16], dz=P[17], dbi=P[18], dS0=P[19], ws=P[20], n=1 << 29, **kw):
        return lib.efla_scan_bwd(ctypes.byref(shape(**kw)), off, u, dl, A, Bm, C, sk, z, bi, S0, dy, dS, du, dd, dA, dB, dC, dsk, dz, dbi, dS0,
                                 ws, n, None)

    for n in ("u", "dl", "A", "Bm", "C", "dy", "du", "dd", "dA", "dB", "dC"):
        assert bwd(**{n: None}) == 1, n
    assert bwd(z=None) == 1 and bwd(dz=None) == 1 and bwd(sk=None) == 1 and bwd(bi=None) == 1
    assert bwd(du=P[0]) == 1 and bwd(dd=P[11]) == 1 and bwd(dA=P[2]) == 1 and bwd(dS0=P[10]) == 1 and bwd(dC=P[14]) == 1 and bwd(ws=P[13]) == 1
    assert bwd(dB=P[14] + 1) == 3 and bwd(dA=P[13] + 2) == 3 and bwd(dS=P[10] + 4) == 3 and bwd(ws=P[20] + 8) == 3
    assert bwd(ws=None) == 4 and bwd(n=64) == 4
    # du, ddelta and dz as slices of one buffer's token rows are apart; shifted by one element they are not
    # (a refused workspace proves that the aliasing check passed: it comes first)
    st = {k + "_s": (19200, 192) for k in ("du", "ddelta", "dz")}
    assert bwd(dd=P[11] + 128, dz=P[11] + 256, ws=None, **st) == 4
    assert bwd(dd=P[11] + 126, dz=P[11] + 256, ws=None, **st) == 1
    assert lib.efla_scan_bwd_workspace_size(ctypes.byref(shape())) > 0
    assert lib.efla_scan_bwd_workspace_size(ctypes.byref(shape(N=65))) == 0
