"""Calls of the scan and the norms that several host threads make at the same time."""
import ctypes
import threading
from functools import partial

import pytest
import torch

import exact_flow_recurrence_gb300 as efla

DEV = "cuda"


def at_once(*calls, times=20000):
    """Each C call from a thread of its own, `times` times: the last errors other than success."""
    codes, start = [0] * len(calls), threading.Barrier(len(calls))

    def loop(i):
        call = calls[i]
        start.wait()
        for _ in range(times):
            rc = call()
            if rc:
                codes[i] = rc

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    efla.efla_get_status()
    return codes


def norm(D):
    """The C call of a norm of D columns, its arguments at hand."""
    x, r, y, h = (torch.randn(4, D, device=DEV) for _ in range(4))
    w, rstd, s = torch.rand(D, device=DEV), torch.empty(4, device=DEV), torch.cuda.Stream()
    shape = efla.RmsShape(rows=4, D=D, x_stride=D, residual_stride=D, y_stride=D, h_stride=D, dtype=efla.F32, weight_dtype=efla.F32, eps=1e-5)
    args = [ctypes.byref(shape)] + [ctypes.c_void_p(t.data_ptr()) for t in (x, r, w, y)] + [None] + [ctypes.c_void_p(t.data_ptr()) for t in (h, rstd)]
    return partial(efla.load_library().efla_rms_fwd, *args, ctypes.c_void_p(s.cuda_stream)), (x, r, y, h, w, rstd, s, shape)


def step(N):
    """... and of a batch's token with N states."""
    B, D = 1300, 96
    u, y, S = torch.randn(B, D, device=DEV), torch.empty(B, D, device=DEV), torch.zeros(B, D, N, device=DEV)
    A, bc, s = -torch.rand(D, N, device=DEV), torch.randn(B, 1, N, device=DEV), torch.cuda.Stream()
    shape = efla.ScanShape(B=B, L=1, D=D, G=1, N=N, dtype=efla.F32, softplus=1)
    for n in ("u", "delta", "y"):
        getattr(shape, n + "_stride")[0] = D
    for n in ("B", "C"):
        getattr(shape, n + "_stride")[0] = N
    p = [ctypes.c_void_p(t.data_ptr()) for t in (u, u, A, bc, bc)] + [None] * 3 + [ctypes.c_void_p(S.data_ptr()), None, B, ctypes.c_void_p(y.data_ptr())]
    return partial(efla.load_library().efla_scan_step, ctypes.byref(shape), *p, ctypes.c_void_p(s.cuda_stream)), (u, y, S, A, bc, s, shape)


@pytest.mark.gpu
@pytest.mark.parametrize("make,sizes", [(norm, (8200, 16384)), (step, (4, 64))])
def test_two_sizes_of_one_kernel_at_once(make, sizes):
    """Two amounts of shared memory: neither call narrows what the other may use."""
    made = [make(n) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert at_once(*(call for call, _ in made)) == [0] * len(made)


def layer_norm(D):
    """... and of a layer norm."""
    x, y = torch.randn(4, D, device=DEV), torch.empty(4, D, device=DEV)
    w, stats, s = torch.rand(D, device=DEV), torch.empty(4, 2, device=DEV), torch.cuda.Stream()
    shape = efla.NormShape(rows=4, D=D, x_stride=D, y_stride=D, dtype=efla.F32, weight_dtype=efla.F32, eps=1e-5)
    args = [ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(w.data_ptr()), None, ctypes.c_void_p(y.data_ptr()), ctypes.c_void_p(stats.data_ptr())]
    return partial(efla.load_library().efla_norm_fwd, ctypes.byref(shape), *args, ctypes.c_void_p(s.cuda_stream)), (x, y, w, stats, s, shape)


@pytest.mark.gpu
def test_two_layer_norms_at_once():
    made = [layer_norm(n) for n in (8200, 16384) for _ in range(2)]
    torch.cuda.synchronize()
    assert at_once(*(call for call, _ in made)) == [0] * len(made)
