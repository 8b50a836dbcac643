"""The gated rule's forward forms that the other tests' sizes do not reach: preparation and scan in one
launch (few heads, at least 640 chunks of a head in all), the tensor cores on a few tokens, and the recurrence past its rule.
Bounds as in test_gated."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from oracle import gated as og
from parity import TOL_F32, assert_close
from test_gated import BF, DEV, F32, check_fwd, draw, gpu, ref64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [efla.EULER, efla.EXACT])
@pytest.mark.parametrize("shape", [(1, 20, 20, 2100, 128, 128), (2, 20, 10, 1151, 64, 64), (1, 48, 48, 1000, 112, 32)])
def test_one_launch(shape, mode):
    x = draw(*shape, BF, mode, rate=0.05, seed=11, token_first=True)
    want = (og.fwd(*(x[n].double() for n in ("q", "k", "v", "g", "beta", "S0")), exact=mode == efla.EXACT), None)
    check_fwd(x, mode, efla.TENSOR, F32, want)
    check_fwd(x, mode, efla.TENSOR, None, want)
    y = gpu(x)
    o, S = efla.efla_gated_fwd(*(y[n] for n in ("q", "k", "v", "g", "beta", "S0")), mode=mode, want_state=False)
    efla.efla_get_status()
    assert S is None
    assert_close("o", o, want[0][0], TOL_F32, stored_bf16=True)
    check_fwd(x, mode, efla.SIMT, F32, want)


def test_one_launch_packed_and_repeated():
    """Sequences of unequal lengths, one empty; the same call twice and in a graph gives the same bits."""
    ends = [0, 700, 700, 701, 2400]
    x = draw(1, 16, 8, 2400, 128, 32, BF, efla.EULER, rate=0.05, seed=12)
    y = {n: t[0] for n, t in gpu(x).items()}
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    gen = torch.Generator().manual_seed(13)
    S0 = torch.randn(4, 16, 128, 32, generator=gen).to(DEV)
    args = [y[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = efla.efla_gated_fwd(*args, S0, offsets=off, out_dtype=F32)
    efla.efla_get_status()
    for b in range(4):
        part = [x[n][:, :, ends[b]:ends[b + 1]].double() for n in ("q", "k", "v", "g", "beta")]
        o_ref, S_ref = og.fwd(*part, S0[b:b + 1].cpu().double())
        assert_close("S_final", S[b:b + 1], S_ref, TOL_F32)
        if ends[b + 1] > ends[b]:
            assert_close("o", o[None, :, ends[b]:ends[b + 1]], o_ref, TOL_F32)
    out = torch.empty_like(o), torch.empty_like(S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        efla.efla_gated_fwd(*args, S0, offsets=off, out_dtype=F32, o=out[0], S_final=out[1])
    for _ in range(2):
        out[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], o) and torch.equal(out[1], S)
    efla.efla_get_status()


@pytest.mark.parametrize("L", [1, 3, 31])
def test_few_tokens_on_the_tensor_cores(L):
    x = draw(2, 2, 1, L, 64, 48, BF, efla.EULER, seed=L)
    want = ref64(x, efla.EULER)
    check_fwd(x, efla.EULER, efla.TENSOR, F32, want)
    check_fwd(x, efla.EULER, efla.TENSOR, None, want)
