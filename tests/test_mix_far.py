"""Elements of the convolution's, the scan's and the RMS norm's arrays that lie past 2^31 of the first: the same values as close by."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
FAR = (1 << 31) + 4096


def far_tokens(t):
    """t [B, L, ...] with its last token more than 2^31 elements behind its first (the memory between them is not touched)."""
    B, L, n = t.shape[0], t.shape[1], t[0, 0].numel()
    step = -(-FAR // (B * L - 1) // 8) * 8
    out = torch.empty(step * (B * L - 1) + n, dtype=t.dtype, device=DEV).as_strided(
        t.shape, (L * step, step) + tuple(t[0, 0].stride()))
    return out.copy_(t)


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_convolution():
    B, L, D = 2, 40, 72
    x, dy, w = torch.randn(B, L, D, device=DEV).to(BF), torch.randn(B, L, D, device=DEV).to(BF), torch.randn(D, 4, device=DEV)
    want = efla.efla_conv_fwd(x, w) + efla.efla_conv_bwd(x, w, dy)
    fx, fy, fdx = far_tokens(x), far_tokens(torch.zeros_like(x)), far_tokens(torch.zeros_like(x))
    got = efla.efla_conv_fwd(fx, w, y=fy) + efla.efla_conv_bwd(fx, w, far_tokens(dy), dx=fdx)
    efla.efla_get_status()
    assert all(torch.equal(p, q) for p, q in zip(got, want) if p is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [40, 300])
def test_scan(L):
    B, D, N = 2, 64, 16
    u, delta, z, dy = (torch.randn(B, L, D, device=DEV).to(BF) for _ in range(4))
    bc, A = torch.randn(2, B, L, 1, N, device=DEV).to(BF), -torch.rand(D, N, device=DEV)
    want = efla.efla_scan_fwd(u, delta, A, *bc, None, z) + efla.efla_scan_bwd(u, delta, A, *bc, dy, None, z)
    fu, fd, fz, fg = (far_tokens(t) for t in (u, delta, z, dy))
    fb, fc = (far_tokens(t) for t in bc)
    outs = [far_tokens(torch.zeros_like(u)) for _ in range(4)]
    got = efla.efla_scan_fwd(fu, fd, A, fb, fc, None, fz, y=outs[0])
    got += efla.efla_scan_bwd(fu, fd, A, fb, fc, fg, None, fz, du=outs[1], ddelta=outs[2], dz=outs[3])
    efla.efla_get_status()
    assert all(torch.equal(p, q) for p, q in zip(got, want) if p is not None)


@pytest.mark.gpu
def test_norm():
    D = 264
    x, r, dy, dh = (torch.randn(1, 50, D, device=DEV).to(BF) for _ in range(4))
    w = torch.rand(D, device=DEV)
    y, _, h, rstd = efla.efla_rms_fwd(x[0], w, r[0])
    q, s, _, _ = efla.efla_rms_fwd(x[0], w, r[0], group=128)
    dx, dw = efla.efla_rms_bwd(h, w, dy[0], rstd, dh=dh[0])
    fx, fr, fy, fh, fdx, fg, fdh = (far_tokens(t)[0] for t in (x, r, torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), dy, dh))
    efla.efla_rms_fwd(fx, w, fr, y=fy, h=fh)
    q2, s2, _, _ = efla.efla_rms_fwd(fx, w, fr, h=fh, group=128, y=far_tokens(torch.zeros_like(q)[None])[0])
    _, dw2 = efla.efla_rms_bwd(fh, w, fg, rstd, dh=fdh, dx=fdx)
    efla.efla_get_status()
    assert torch.equal(fy, y) and torch.equal(fh, h) and torch.equal(fdx, dx) and torch.equal(dw2, dw) and torch.equal(s2, s)
    assert torch.equal(q2.contiguous().view(torch.uint8), q.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 700])
def test_steps_on_a_long_cache(B):
    """(700 sequences: the ring of a batch.)"""
    D, N, W = 4096, 16, 4
    n = FAR // (D * N) + 2
    S = torch.empty(n, D, N, device=DEV)
    near = torch.randn(B, D, N, device=DEV)
    slots = torch.arange(n - 1, n - 1 - B, -1, dtype=torch.int32, device=DEV)
    S[slots.long()] = near
    u, delta = torch.randn(B, D, device=DEV).to(BF), torch.randn(B, D, device=DEV).to(BF)
    bc, A = torch.randn(B, 1, N, device=DEV).to(BF), -torch.rand(D, N, device=DEV)
    want = efla.efla_scan_step(u, delta, A, bc, bc, near)
    got = efla.efla_scan_step(u, delta, A, bc, bc, S, slots=slots)
    efla.efla_get_status()
    assert torch.equal(got, want) and torch.equal(S[slots.long()], near)
    del S
    n = FAR // ((W - 1) * D) + 2
    C = torch.empty(n, W - 1, D, dtype=BF, device=DEV)
    near, w = torch.randn(B, W - 1, D, device=DEV).to(BF), torch.randn(D, W, device=DEV)
    slots = torch.arange(n - 1, n - 1 - B, -1, dtype=torch.int32, device=DEV)
    C[slots.long()] = near
    want = efla.efla_conv_step(u, w, near)
    got = efla.efla_conv_step(u, w, C, slots=slots)
    efla.efla_get_status()
    assert torch.equal(got, want) and torch.equal(C[slots.long()], near)
