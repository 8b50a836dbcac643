"""A token-mixing block on the gated operators: layer norm, projections, gated delta rule, output.

    x + Wo . gated_delta_rule(q, k, v, g, beta),   q, k, v, beta, g from layer_norm(x)

Training runs the norm and the rule, forward and backward, as autograd functions.  Serving runs
several prompts of unequal lengths packed on one axis of tokens, keeps each sequence's state in a
cache, and goes on a token at a time with the decode step.  Run it on one GPU:

    python -m examples.gated_block
"""
import math

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

import exact_flow_recurrence_gb300 as efla

DK = 128   # a head's size


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, stats = efla.efla_norm_fwd(x, weight, bias)
        ctx.save_for_backward(x, weight, stats)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, stats = ctx.saved_tensors
        return efla.efla_norm_bwd(x, weight, dy.contiguous(), stats)


class GatedRule(torch.autograd.Function):
    """The rule from a zero state; alpha as in the exact flow (any key length is stable)."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return efla.efla_gated_fwd(q, k, v, g, beta, mode=efla.EXACT, want_state=False)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        if dO.stride(-1) != 1 or 0 in dO.stride():   # broadcast, as the gradient of a sum is
            dO = dO.contiguous()
        return efla.efla_gated_bwd(*ctx.saved_tensors, dO, mode=efla.EXACT, want_dS0=False)[:5]


class GatedBlock:
    """Weights of one block with H heads on rows of D values (bf16; the norm's and gate's in fp32)."""

    def __init__(self, D: int, H: int, device, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)

        def draw(*shape):
            return (torch.randn(*shape, generator=gen) / math.sqrt(shape[-1])).to(device, torch.bfloat16).requires_grad_()

        self.D, self.H = D, H
        self.w_norm = torch.ones(D, device=device).requires_grad_()
        self.b_norm = torch.zeros(D, device=device).requires_grad_()
        self.w_in = draw(3 * H * DK + H, D)      # q, k, v, beta
        self.w_gate = draw(H, D)                 # the decay
        self.b_gate = torch.linspace(-6.0, 0.0, H).to(device).requires_grad_()   # memories from long to short
        self.w_out = draw(D, H * DK)

    def parameters(self):
        return [self.w_norm, self.b_norm, self.w_in, self.w_gate, self.b_gate, self.w_out]

    def _decay(self, y):   # log decay, <= 0
        return -F.softplus((y @ self.w_gate.t()).float() + self.b_gate)

    def _project(self, y):
        """y [..., D] -> q, k, v [..., H, dk] (k, v as they lie in the projection's output) and beta, g [..., H]."""
        H = self.H
        p = y @ self.w_in.t()
        heads = p[..., : 3 * H * DK].unflatten(-1, (3, H, DK))
        beta = torch.sigmoid(p[..., 3 * H * DK:].float())
        return heads[..., 0, :, :] * (1 / math.sqrt(DK)), heads[..., 1, :, :], heads[..., 2, :, :], beta, self._decay(y)

    def train_forward(self, x):
        """x [B, L, D] bf16 -> the block's output; differentiable."""
        B, L, _ = x.shape
        q, k, v, beta, g = self._project(LayerNorm.apply(x, self.w_norm, self.b_norm))
        # heads first, as views: the operators take strided heads
        o = GatedRule.apply(*(t.transpose(1, 2) for t in (q, k, v)), g.transpose(1, 2), beta.transpose(1, 2))
        return x + o.transpose(1, 2).reshape(B, L, self.H * DK) @ self.w_out.t()

    @torch.no_grad()
    def prefill(self, x, offsets, cache, slots):
        """Packed prompts x [T, D], offsets int32 [B + 1]; their states go to cache[slots]."""
        q, k, v, beta, g = self._project(efla.efla_norm_fwd(x, self.w_norm, self.b_norm)[0])
        o, S = efla.efla_gated_fwd(*(t.transpose(0, 1) for t in (q, k, v, g, beta)), offsets=offsets, mode=efla.EXACT)
        cache.index_copy_(0, slots.long(), S)
        return x + o.transpose(0, 1).reshape(-1, self.H * DK) @ self.w_out.t()

    @torch.no_grad()
    def decode(self, x, cache, slots):
        """One token of each sequence, x [B, D]; cache[slots] moves on in place."""
        q, k, v, beta, g = self._project(efla.efla_norm_fwd(x, self.w_norm, self.b_norm)[0])
        o = efla.efla_gated_step(q, k, v, g, beta, cache, slots=slots, mode=efla.EXACT)
        return x + o.reshape(-1, self.H * DK) @ self.w_out.t()


def main():
    dev = torch.device("cuda:0")
    D, H = 1024, 8
    block = GatedBlock(D, H, dev)
    gen = torch.Generator().manual_seed(1)

    # training: a few steps towards giving out the token before
    opt = torch.optim.Adam(block.parameters(), lr=1e-3)
    for it in range(20):
        x = torch.randn(4, 512, D, generator=gen).to(dev, torch.bfloat16)
        loss = F.mse_loss(block.train_forward(x)[:, 1:].float(), x[:, :-1].float())
        opt.zero_grad()
        loss.backward()
        opt.step()
        if it % 5 == 4:
            print(f"step {it + 1}: loss {loss.item():.4f}")

    # serving: three prompts, their states at places 5, 0 and 3 of a cache of 8, then eight tokens more
    lens = [300, 1, 77]
    offsets = torch.tensor([0, 300, 301, 378], dtype=torch.int32, device=dev)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device=dev)
    cache = torch.zeros(8, H, DK, DK, device=dev)
    x = torch.randn(sum(lens), D, generator=gen).to(dev, torch.bfloat16)
    out = block.prefill(x, offsets, cache, slots)
    token = out[(offsets[1:] - 1).long()]
    for _ in range(8):
        token = block.decode(token, cache, slots)
    efla.efla_get_status()
    print("served", len(lens), "sequences; |state|:", [f"{cache[s].norm().item():.2f}" for s in slots.tolist()])


if __name__ == "__main__":
    main()
