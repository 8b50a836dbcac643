"""The gated rule's tensor-core kernels and the batched step through the debug library: every checked
write lands in its buffer, and the results are the release library's bit for bit."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from test_debug_build import _same, _with
from test_debug_build import libs  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _draw(B, H, Hk, L, dk, dv, packed, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def rnd(*shape, t=torch.bfloat16):
        return torch.randn(*shape, generator=gen).to(DEV, t)

    lead = () if packed else (B,)
    q, k = rnd(*lead, Hk, L, dk), (rnd(*lead, Hk, L, dk).float() / dk ** 0.5).bfloat16()
    v, dO = rnd(*lead, H, L, dv), rnd(*lead, H, L, dv)
    g = -0.1 * torch.rand(*lead, H, L, generator=gen).to(DEV)
    beta = torch.rand(*lead, H, L, generator=gen).to(DEV)
    S0, dS = rnd(B, H, dk, dv, t=torch.float32), rnd(B, H, dk, dv, t=torch.float32)
    off = torch.tensor([0] + [L * (b + 1) * (b + 2) // (B * (B + 1)) for b in range(B)], dtype=torch.int32).to(DEV)
    return q, k, v, g, beta, dO, S0, dS, off if packed else None


@pytest.mark.parametrize("sizes", [(2, 4, 2, 200, 128, 128, False), (3, 2, 2, 333, 64, 96, True), (1, 80, 80, 130, 48, 64, False),
                                   (1, 20, 10, 2100, 128, 128, False)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gated(libs, sizes, out):  # noqa: F811
    q, k, v, g, beta, dO, S0, dS, off = _draw(*sizes)
    rel, dbg = libs
    for fn in (lambda: efla.efla_gated_fwd(q, k, v, g, beta, S0, offsets=off, out_dtype=out, path=efla.TENSOR),
               lambda: efla.efla_gated_fwd(q, k, v, g, beta, offsets=off, out_dtype=out, want_state=False, path=efla.TENSOR),
               lambda: efla.efla_gated_bwd(q, k, v, g, beta, dO, S0, dS, offsets=off, out_dtype=out, path=efla.TENSOR)):
        _same(_with(rel, fn), _with(dbg, fn))


def test_step(libs):  # noqa: F811
    q, k, v, g, beta, _, S0, _, _ = _draw(40, 8, 4, 1, 128, 128, False)

    def fn():
        S = S0.clone()
        return efla.efla_gated_step(*(t[:, :, 0] for t in (q, k, v, g, beta)), S), S

    rel, dbg = libs
    _same(_with(rel, fn), _with(dbg, fn))
