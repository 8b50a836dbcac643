"""The short causal convolution at lengths that keep a thread walking: runs of up to 128 tokens, several of them a sequence, ends
of packed sequences inside them; against the same formulas over whole tensors in 64 bits.  max |err| / rms <= 1e-5: a value
is W + 1 products and sums (2^-24 of each), then a sigmoid of relative error (1.3 |x| + 8) 2^-24, at most 1.8e-6 at the |x| <= 16
met here.  dw and db add a run's 128 terms at most one after another (sqrt(128) 2^-24 of their rms at random), eight runs of a
CTA, then the CTAs' sums in eight groups of rows: under 5e-6.  Values stored in bf16 add half an ulp."""
import random

import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from parity import assert_close

TOL = 1e-5
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def reference(seqs, x, w, b, S0, dy, dS, silu):
    """(y, S_final, dx, dw, db, dS0) of sequences [a, e) of x [T, D], all in fp64 on the GPU."""
    D, W = w.shape
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    last, dS0 = torch.zeros_like(S0), torch.zeros_like(S0)
    dw, db = torch.zeros_like(w), torch.zeros(D, dtype=x.dtype, device=x.device)
    for i, (a, e) in enumerate(seqs):
        n = e - a
        rows = torch.cat([S0[i], x[a:e]])
        last[i] = rows[n:]
        pre = sum(w[:, j] * rows[j:j + n] for j in range(W)) + (0 if b is None else b)
        sig = torch.sigmoid(pre)
        y[a:e] = pre * sig if silu else pre
        dp = dy[a:e] * sig * (1 + pre * (1 - sig)) if silu else dy[a:e]
        dr = torch.zeros_like(rows)
        dr[n:] += dS[i]
        for j in range(W):
            dr[j:j + n] += w[:, j] * dp
            dw[:, j] += (dp * rows[j:j + n]).sum(0)
        db += dp.sum(0)
        dS0[i], dx[a:e] = dr[:W - 1], dr[W - 1:]
    return y, last, dx, dw, db, dS0


def check(B, L, D, W, dtype, lens=None, silu=True, bias=True, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + D + L)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    packed = lens is not None
    ends = [0]
    for n in lens if packed else [L] * B:
        ends.append(ends[-1] + n)
    n, T = len(ends) - 1, ends[-1]
    lead = (T,) if packed else (B, L)
    x, dy = rnd(*lead, D).to(dtype), rnd(*lead, D).to(dtype)
    w, b = rnd(D, W) / 2, 0.2 * rnd(D) if bias else None
    S0, dS = rnd(n, W - 1, D).to(dtype), rnd(n, W - 1, D).to(dtype)
    off = torch.tensor(ends, dtype=torch.int32, device=DEV) if packed else None
    y, last = efla.efla_conv_fwd(x, w, b, S0, offsets=off, silu=silu)
    got = efla.efla_conv_bwd(x, w, dy, b, S0, dS, offsets=off, silu=silu)
    efla.efla_get_status()
    ref = reference(list(zip(ends, ends[1:])), x.double().view(T, D), w.double(), b.double() if bias else None, S0.double(),
                    dy.double().view(T, D), dS.double(), silu)
    bf = dtype == BF
    assert_close("y", y.view(T, D), ref[0], TOL, stored_bf16=bf)
    assert torch.equal(last.double(), ref[1])
    assert_close("dx", got[0].view(T, D), ref[2], TOL, stored_bf16=bf)
    assert_close("dw", got[1], ref[3], TOL)
    if bias:
        assert_close("db", got[2], ref[4], TOL)
    assert_close("dS0", got[3], ref[5], TOL, stored_bf16=bf)
    again = efla.efla_conv_bwd(x, w, dy, b, S0, dS, offsets=off, silu=silu)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,L,D,W", [(8, 2048, 2048, 4), (4, 2047, 1025, 4), (4, 2047, 1025, 3), (3, 4001, 1024, 2), (2, 6007, 513, 2)])
def test_long_runs(B, L, D, W, dtype):
    check(B, L, D, W, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,W", [(2048, 4), (1001, 3), (1536, 2)])
def test_packed_ends_inside_runs(D, W, dtype):
    """Some 16000 tokens: long sequences, many short ones, empty ones, ends at every place of a run."""
    r = random.Random(D)
    lens = [3001, 0, 1, 2, 3, 997] + [r.randint(0, 40) for _ in range(150)] + [5003, 1, 0, 0, 2500] + [r.randint(1, 9) for _ in range(60)] + [999]
    check(0, 0, D, W, dtype, lens=lens, bias=W != 3, silu=W != 2)
