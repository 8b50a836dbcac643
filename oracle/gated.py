"""64-bit reference of the gated delta rule and of layer norm, for the tests.

Token by token, from the definitions, in fp64 on the CPU:
    S <- e^{g_t} S,   S <- S + alpha_t k_t (v_t - S^T k_t)^T,   o_t = S^T q_t
with alpha_t = beta_t, or (1 - e^{-beta_t lambda_t}) / lambda_t with lambda_t = ||k_t||^2.
Gradients by automatic differentiation of the same loop.
"""
from __future__ import annotations

import torch


def alpha(k, beta, exact: bool):
    if not exact:
        return beta
    x = beta * (k * k).sum(-1)
    # -expm1(-x)/x, continued by its series at 0 (the quotient and its derivative are 0/0 there)
    small = x.abs() < 1e-4
    safe = torch.where(small, torch.ones_like(x), x)
    return beta * torch.where(small, 1 - x / 2 + x * x / 6 - x ** 3 / 24, -torch.expm1(-safe) / safe)


def fwd(q, k, v, g, beta, S0=None, exact: bool = False):
    """q, k [B,Hk,L,dk], v [B,H,L,dv], g, beta [B,H,L], S0 [B,H,dk,dv] or None, fp64: (o, S_final)."""
    B, H, L, dv = v.shape
    rep = H // k.shape[1]
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    a = alpha(k, beta, exact)
    S = torch.zeros(B, H, k.shape[-1], dv, dtype=torch.float64) if S0 is None else S0
    o = []
    for t in range(L):
        S = S * torch.exp(g[:, :, t])[..., None, None]
        r = v[:, :, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, :, t])
        S = S + (a[:, :, t, None] * k[:, :, t])[..., None] * r[..., None, :]
        o.append(torch.einsum("bhkv,bhk->bhv", S, q[:, :, t]))
    return (torch.stack(o, 2) if o else torch.zeros_like(v)), S


def bwd(q, k, v, g, beta, dO, S0=None, dS_final=None, exact: bool = False):
    """Gradients of sum(o dO) + sum(S_final dS_final): (dq, dk, dv, dg, dbeta, dS0)."""
    S0 = torch.zeros(*v.shape[:2], k.shape[-1], v.shape[-1], dtype=torch.float64) if S0 is None else S0
    leaf = [x.detach().clone().requires_grad_() for x in (q, k, v, g, beta, S0)]
    o, S = fwd(*leaf, exact=exact)
    loss = (o * dO).sum() + (0 * S if dS_final is None else S * dS_final).sum()
    grads = torch.autograd.grad(loss, leaf, allow_unused=True)
    return tuple(torch.zeros_like(x) if d is None else d for x, d in zip(leaf, grads))


def norm_fwd(x, w, b, eps: float):
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mean) * rstd * w
    return (y if b is None else y + b), torch.cat([mean, rstd], -1)


def norm_bwd(x, w, dy, eps: float):
    """(dx, dw, db) of sum(y dy)."""
    leaf = [t.detach().clone().requires_grad_() for t in (x, w, torch.zeros_like(w))]
    y, _ = norm_fwd(*leaf, eps)
    return torch.autograd.grad((y * dy).sum(), leaf)
