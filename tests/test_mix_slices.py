"""Inputs and outputs that are slices of one buffer's token rows."""
import ctypes

import pytest
import torch

import exact_flow_recurrence_gb300 as efla

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 37])
def test_steps_from_and_into_one_buffer(D, dtype):
    """One token a sequence: x (or u, delta, B and C) beside y in the rows of a projection."""
    B, N, W = 5, 8, 4
    rows = torch.randn(B, 3 * D + 2 + N, device=DEV).to(dtype)
    x, delta, y = (rows[:, i * D:(i + 1) * D] for i in range(3))
    w, S = torch.randn(D, W, device=DEV), torch.randn(B, W - 1, D, device=DEV).to(dtype)
    want = efla.efla_conv_step(x.contiguous(), w, S.clone())
    assert efla.efla_conv_step(x, w, S, y=y) is y
    efla.efla_get_status()
    assert torch.equal(y, want)
    A, bc, S = -torch.rand(D, N, device=DEV), rows[:, None, 3 * D + 2:], torch.randn(B, D, N, device=DEV)
    keep = rows.clone()
    want = efla.efla_scan_step(x.contiguous(), delta.contiguous(), A, bc.contiguous(), bc.contiguous(), S.clone())
    efla.efla_scan_step(x, delta, A, bc, bc, S, y=y)
    efla.efla_get_status()
    assert torch.equal(y, want) and torch.equal(rows[:, :2 * D], keep[:, :2 * D]) and torch.equal(rows[:, 3 * D:], keep[:, 3 * D:])


@pytest.mark.gpu
@pytest.mark.parametrize("time_major", [False, True])
@pytest.mark.parametrize("L", [1, 9])
def test_sequences_from_and_into_one_buffer(L, time_major):
    B, D = 3, 64
    rows = torch.randn(L, B, 2 * D, device=DEV).transpose(0, 1) if time_major else torch.randn(B, L, 2 * D, device=DEV)
    x, y, w = rows[..., :D], rows[..., D:], torch.randn(D, 4, device=DEV)
    want = efla.efla_conv_fwd(x.contiguous(), w)[0]
    efla.efla_conv_fwd(x, w, y=y)
    efla.efla_get_status()
    assert torch.equal(y, want)


def test_steps_into_rows_that_share_elements_are_refused():
    """Host checks: nothing is launched (no GPU needed)."""
    lib, p = efla.load_library(), [0x7f0000000000 + i * 0x40000000 for i in range(4)]

    def step(y, x_stride, y_stride):
        s = efla.ConvShape(B=4, L=1, D=64, W=4, dtype=efla.BF16, weight_dtype=efla.F32)
        s.x_stride[0], s.y_stride[0] = x_stride, y_stride
        return lib.efla_conv_step(ctypes.byref(s), p[0], p[1], None, p[2], None, 4, y, None)

    def bwd(dx, x_stride, dx_stride):
        """(A refused workspace, 4, proves that the aliasing check passed: it comes first.)"""
        s = efla.ConvShape(B=4, L=10, D=64, W=4, dtype=efla.BF16, weight_dtype=efla.F32)
        for n, st in (("x", x_stride), ("dy", (640, 64)), ("dx", dx_stride)):
            setattr(s, n + "_stride", type(s.x_stride)(*st))
        return lib.efla_conv_bwd(ctypes.byref(s), None, p[0], p[1], None, None, p[2], None, dx, p[3], None, None, None, 0, None)

    for st in ((1280, 128), (128, 512)):      # batch-major and time-major rows of 128
        assert bwd(p[0] + 128, st, st) == 4
        assert bwd(p[0] + 126, st, st) == 1 and bwd(p[0], st, st) == 1
    assert bwd(p[0] + 128, (128, 512), (1280, 128)) == 1 and bwd(p[0] + 128, (128, 500), (128, 500)) == 1
    assert bwd(p[0] + 128, (100, 1000), (100, 1000)) == 1
    assert step(p[0] + 126, 128, 128) == 1 and step(p[0], 128, 128) == 1 and step(p[0] + 128, 96, 96) == 1
    assert step(p[0] + 128, 128, 256) == 1 and step(p[3], 128, 32) == 1
