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
