"""64-bit reference of the short causal convolution, the selective scan and the residual's RMS norm, for the tests.

From the definitions, token by token, in fp64 on the CPU; gradients by automatic differentiation of the same loops.
A sequence is [L, ...]; `over` runs several, packed on one axis or as a batch.
"""
from __future__ import annotations

import torch


def conv(x, w, b, S0, silu: bool):
    """x [L,D], w [D,W], b [D] or None, S0 [W-1,D] or None: (y [L,D], the last W - 1 rows)."""
    wide = w.shape[1] - 1
    rows = torch.cat([torch.zeros(wide, x.shape[1], dtype=x.dtype) if S0 is None else S0, x])
    y = []
    for t in range(x.shape[0]):
        pre = (rows[t:t + wide + 1] * w.t()).sum(0)
        pre = pre if b is None else pre + b
        y.append(pre * torch.sigmoid(pre) if silu else pre)
    return (torch.stack(y) if y else torch.zeros_like(x)), rows[x.shape[0]:]


def scan(u, delta, A, B, C, D, z, dbias, S0, softplus: bool):
    """u, delta, z [L,Di], A [Di,N], B, C [L,G,N], D, dbias [Di], S0 [Di,N]: (y [L,Di], the last state)."""
    h = torch.zeros_like(A) if S0 is None else S0
    rep = A.shape[0] // B.shape[1]
    raw = delta if dbias is None else delta + dbias
    dt = torch.nn.functional.softplus(raw, threshold=50) if softplus else raw
    y = []
    for t in range(u.shape[0]):
        h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * u[t])[:, None] * B[t].repeat_interleave(rep, 0)
        o = (h * C[t].repeat_interleave(rep, 0)).sum(-1)
        o = o if D is None else o + D * u[t]
        y.append(o if z is None else o * z[t] * torch.sigmoid(z[t]))
    return (torch.stack(y) if y else torch.zeros_like(u)), h


def over(seqs, fn, tokens, shared, states):
    """fn(*tokens of a sequence, *shared, its state) for each (start, end) of the packed axis: (outputs, last states)."""
    ys, last = [], []
    for i, (a, b) in enumerate(seqs):
        y, s = fn([None if t is None else t[a:b] for t in tokens], shared, None if states is None else states[i])
        ys.append(y)
        last.append(s)
    return torch.cat(ys), torch.stack(last)


def conv_all(seqs, x, w, b, S0, silu):
    return over(seqs, lambda t, s, S: conv(t[0], s[0], s[1], S, silu), [x], (w, b), S0)


def scan_all(seqs, u, delta, A, B, C, D, z, dbias, S0, softplus):
    return over(seqs, lambda t, s, S: scan(t[0], t[1], s[0], t[2], t[3], s[1], t[4], s[2], S, softplus),
                [u, delta, B, C, z], (A, D, dbias), S0)


def grads(fn, args, dy, dS):
    """Gradients of sum(y dy) + sum(S dS) with respect to every tensor of args; None for the others."""
    leaf = [a.detach().clone().requires_grad_() if torch.is_tensor(a) else a for a in args]
    y, S = fn(*leaf)
    loss = (y * dy).sum() + (0 * S if dS is None else S * dS).sum() + sum(0 * a.sum() for a in leaf if torch.is_tensor(a))
    at = [i for i, a in enumerate(leaf) if torch.is_tensor(a)]
    got = torch.autograd.grad(loss, [leaf[i] for i in at], allow_unused=True)
    out = [None] * len(args)
    for i, g in zip(at, got):
        out[i] = torch.zeros_like(leaf[i]) if g is None else g
    return out


def rms_fwd(h, w, eps: float):
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h * rstd[..., None] * w, rstd


def rms_bwd(h, w, dy, eps: float, dh=None):
    """(dx, dw) of sum(y dy) + sum(h dh)."""
    leaf = [t.detach().clone().requires_grad_() for t in (h, w)]
    loss = (rms_fwd(*leaf, eps)[0] * dy).sum() + (0 if dh is None else (leaf[0] * dh).sum())
    return torch.autograd.grad(loss, leaf)
