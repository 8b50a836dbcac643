"""Host-side refusals of the gated delta rule's C entry points (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import exact_flow_recurrence_gb300 as efla

A = 0x7f0000000000
P = [A + i * 0x40000000 for i in range(20)]


@pytest.fixture(scope="module")
def lib():
    return efla.load_library()


def shape(**kw):
    a = dict(B=2, H=4, Hk=2, L=100, dk=64, dv=32, dtype=torch.bfloat16)
    tail = {n: kw.pop(n) for n in list(kw) if n not in ("B", "H", "Hk", "L", "dk", "dv", "packed", "strides", "mode", "path")}
    a.update(kw)
    s = efla.make_gated_shape(**a)
    for n, v in tail.items():
        setattr(s, n, v)
    return s


def fwd(lib, s, off=None, q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], S0=None, o=P[5], Sf=None, ws=P[6], n=1 << 29):
    return lib.efla_gated_fwd(ctypes.byref(s), off, q, k, v, g, beta, S0, o, Sf, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=24), 2), (dict(dv=144), 2), (dict(dtype=5), 2), (dict(out_dtype=5), 2), (dict(mode=7), 2), (dict(path=9), 2),
    (dict(B=-1), 1), (dict(L=-1), 1), (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(packed=2), 1), (dict(H=131072, Hk=1), 2),
    (dict(strides={"q": (64, 64, -64)}), 1),
    (dict(strides={"o": (0, 3200, 32)}), 1),        # two sequences write the same rows
    (dict(strides={"o": (12800, 3200, 16)}), 1),    # rows overlap
])
def test_bad_shapes(lib, kw, code):
    s = shape(**kw)
    assert fwd(lib, s) == code and lib.efla_last_error().decode()
    if code == 2 or "strides" not in kw:
        assert lib.efla_gated_fwd_workspace_size(ctypes.byref(s)) == 0


def test_bad_pointers(lib):
    s = shape()
    assert lib.efla_gated_fwd(None, None, *P[:5], None, P[5], None, P[6], 1 << 29, None) == 1
    for n in ("q", "k", "v", "g", "beta", "o"):
        assert fwd(lib, s, **{n: None}) == 1, n
    assert fwd(lib, s, q=P[0] + 1) == 3 and fwd(lib, s, g=P[3] + 2) == 3 and fwd(lib, s, S0=P[7] + 4) == 3
    assert fwd(lib, s, o=P[2]) == 1 and fwd(lib, s, o=P[0] + 64) == 1
    assert fwd(lib, s, Sf=P[2]) == 1 and fwd(lib, s, ws=P[0]) == 1 and fwd(lib, s, ws=P[5]) == 1
    assert fwd(lib, s, S0=P[7], Sf=P[7] + 256) == 1
    assert fwd(lib, s, ws=None) == 4 and fwd(lib, s, n=64) == 4
    assert fwd(lib, shape(packed=True), off=None) == 1
    assert fwd(lib, shape(packed=True), off=P[8] + 2) == 3
    assert fwd(lib, shape(B=0), q=None, k=None, v=None, g=None, beta=None, o=None, ws=None, n=0) == 0


def test_backward_refusals(lib):
    s = shape()

    def bwd(s=s, dO=P[5], dS=None, dq=P[6], dk=P[7], dv=P[8], dg=P[9], db=P[10], dS0=None, ws=P[11], n=1 << 29):
        return lib.efla_gated_bwd(ctypes.byref(s), None, *P[:5], None, dO, dS, dq, dk, dv, dg, db, dS0, ws, n, None)

    assert bwd(dO=None) == 1 and bwd(dq=None) == 1 and bwd(dg=None) == 1
    assert bwd(dk=P[6]) == 1 and bwd(dv=P[2]) == 1 and bwd(db=P[9]) == 1 and bwd(dS0=P[8]) == 1 and bwd(dg=P[0]) == 1
    assert bwd(dg=P[9] + 4) == 3 and bwd(ws=None) == 4 and bwd(n=64) == 4 and bwd(ws=P[9]) == 1
    assert bwd(dS=P[12], dS0=P[12]) == 1
    # dq, dk, dv as slices of one buffer's token rows are apart; shifted by one element they are not
    w = 2 * 64 * 2 + 4 * 32
    st = {n: (100 * w, d, w) for n, d in (("dq", 64), ("dk", 64), ("dv", 32))}
    f = shape(strides=st)
    # (a refused workspace proves that the aliasing check passed: it comes first)
    assert bwd(f, dq=P[6], dk=P[6] + 2 * 128, dv=P[6] + 2 * 256, ws=None) == 4
    assert bwd(f, dq=P[6], dk=P[6] + 2 * 127, dv=P[6] + 2 * 256, ws=None) == 1


def test_step_refusals(lib):
    s = shape(L=1)

    def step(s=s, q=P[0], S=P[5], slots=None, n=2, o=P[6]):
        return lib.efla_gated_step(ctypes.byref(s), q, *P[1:5], S, slots, n, o, None)

    assert step(shape(L=2)) == 1 and step(shape(L=1, packed=True)) == 1 and step(shape(L=1, path=efla.TENSOR)) == 2
    assert step(S=None) == 1 and step(q=None) == 1 and step(n=1) == 1 and step(n=-1) == 1
    assert step(o=P[5]) == 1 and step(S=P[0]) == 1 and step(S=P[5] + 8) == 3 and step(slots=P[7] + 1) == 3
    assert step(slots=P[5]) == 1
    assert step(shape(B=0, L=1), S=None, n=0, o=None, q=None) == 0


def test_workspaces_grow(lib):
    a, b = (lib.efla_gated_bwd_workspace_size(ctypes.byref(shape(L=n))) for n in (64, 1000))
    assert 0 < a < b
    assert lib.efla_gated_fwd_workspace_size(ctypes.byref(shape(L=0))) == 0


def test_tensor_path_needs_bf16_rows_on_16_bytes(lib):
    assert fwd(lib, shape(path=efla.TENSOR, dtype=efla.F32)) == 2
    assert fwd(lib, shape(path=efla.TENSOR), k=P[1] + 2) == 2
    assert fwd(lib, shape(path=efla.TENSOR, strides={"v": (12808, 3200, 36)})) == 2
    assert fwd(lib, shape(path=efla.TENSOR, strides={"q": (12800, 0, 64)})) == 2
    assert fwd(lib, shape(path=efla.TENSOR), ws=None) == 4      # accepted up to its workspace


def test_packed_slots(lib):
    assert lib.efla_gated_fwd_workspace_size(ctypes.byref(shape(L=0, packed=True))) > 0
