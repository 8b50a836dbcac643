"""A selective state space block on the framework's operators: RMS norm of the residual stream, projections, short
convolution, selective scan, output.

    y, h = rms(x + stream);   u, z = halves of Wi y;   u = silu(conv(u));   (r, B, C) = Wx u;   delta = Wd r
    out = Wo . scan(u, delta, A, B, C, D, z, bias)

The block takes what the layer before put out and the stream in front of it, and gives its own output and the stream h, so
that the addition is part of the next norm.  Training runs norm, convolution and scan as autograd functions.  Serving runs
several prompts of unequal lengths packed on one axis of tokens, keeps each sequence's last inputs and states in caches, and
goes on a token at a time.  Run it on one GPU:

    python -m examples.scan_block
"""
import math

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

import exact_flow_recurrence_gb300 as efla

N = 16   # states a channel
W = 4    # taps


def _dense(g):
    """A gradient that the operators read: broadcast ones, as the gradient of a sum is, are written out."""
    return g.contiguous() if g.stride(-1) != 1 or 0 in g.stride() else g


class RmsNorm(torch.autograd.Function):
    """(y, h): the norm of h = x + stream, and h."""

    @staticmethod
    def forward(ctx, x, stream, weight):
        y, _, h, rstd = efla.efla_rms_fwd(x, weight, stream)
        ctx.save_for_backward(h, weight, rstd)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        dx, dw = efla.efla_rms_bwd(h, weight, _dense(dy).contiguous(), rstd, dh=_dense(dh).contiguous())
        return dx, dx, dw


class ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return efla.efla_conv_fwd(x, weight, bias, want_state=False)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        return efla.efla_conv_bwd(x, weight, _dense(dy), bias, want_dS0=False)[:3]


class SelectiveScan(torch.autograd.Function):
    """The scan from a zero state."""

    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, bias):
        ctx.save_for_backward(u, delta, A, B, C, D, z, bias)
        return efla.efla_scan_fwd(u, delta, A, B, C, D, z, bias, want_state=False)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        u, delta, A, B, C, D, z, bias = ctx.saved_tensors
        return efla.efla_scan_bwd(u, delta, A, B, C, _dense(dy), D, z, bias, want_dS0=False)[:8]


class ScanBlock:
    """Weights of one block on rows of D values, with Di channels (bf16; the norm's, convolution's and scan's own in fp32)."""

    def __init__(self, D: int, Di: int, device, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)

        def draw(*shape):
            return (torch.randn(*shape, generator=gen) / math.sqrt(shape[-1])).to(device, torch.bfloat16).requires_grad_()

        self.D, self.Di, self.R = D, Di, max(8, D // 16)
        self.w_norm = torch.ones(D, device=device).requires_grad_()
        self.w_in = draw(2 * Di, D)
        self.w_conv = (torch.randn(Di, W, generator=gen) / math.sqrt(W)).to(device).requires_grad_()
        self.b_conv = torch.zeros(Di, device=device).requires_grad_()
        self.w_x = draw(self.R + 2 * N, Di)
        self.w_dt = draw(Di, self.R)
        size = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(Di, generator=gen))   # step sizes to begin with
        self.b_dt = (size + torch.log(-torch.expm1(-size))).to(device).requires_grad_()
        self.log_A = torch.log(1.0 + torch.arange(N)).expand(Di, N).contiguous().to(device).requires_grad_()
        self.skip = torch.ones(Di, device=device).requires_grad_()
        self.w_out = draw(D, Di)

    def parameters(self):
        return [self.w_norm, self.w_in, self.w_conv, self.b_conv, self.w_x, self.w_dt, self.b_dt, self.log_A, self.skip, self.w_out]

    def _inputs(self, u):
        """delta, B, C (one group; slices of the projection's rows) of the convolution's output."""
        p = u @ self.w_x.t()
        B, C = (p[..., self.R + i * N: self.R + (i + 1) * N].unsqueeze(-2) for i in (0, 1))
        return p[..., : self.R] @ self.w_dt.t(), B, C

    def train_forward(self, x, stream):
        """x, stream [B, L, D] bf16 -> (the block's output, the stream behind its norm); differentiable."""
        y, h = RmsNorm.apply(x, stream, self.w_norm)
        xz = y @ self.w_in.t()
        u = ShortConv.apply(xz[..., : self.Di], self.w_conv, self.b_conv)
        delta, B, C = self._inputs(u)
        o = SelectiveScan.apply(u, delta, -torch.exp(self.log_A), B, C, self.skip, xz[..., self.Di:], self.b_dt)
        return o @ self.w_out.t(), h

    def caches(self, n: int):
        """Room for n sequences: their last inputs, and their states."""
        dev = self.w_in.device
        return torch.zeros(n, W - 1, self.Di, dtype=torch.bfloat16, device=dev), torch.zeros(n, self.Di, N, device=dev)

    @torch.no_grad()
    def prefill(self, x, stream, offsets, caches, slots):
        """Packed prompts x, stream [T, D], offsets int32 [B + 1]; what they leave goes to the caches' places `slots`."""
        y, _, h, _ = efla.efla_rms_fwd(x, self.w_norm, stream)
        xz = y @ self.w_in.t()
        u, rows = efla.efla_conv_fwd(xz[..., : self.Di], self.w_conv, self.b_conv, offsets=offsets)
        delta, B, C = self._inputs(u)
        o, S = efla.efla_scan_fwd(u, delta, -torch.exp(self.log_A), B, C, self.skip, xz[..., self.Di:], self.b_dt, offsets=offsets)
        caches[0].index_copy_(0, slots.long(), rows)
        caches[1].index_copy_(0, slots.long(), S)
        return o @ self.w_out.t(), h

    @torch.no_grad()
    def decode(self, x, stream, caches, slots):
        """One token of each sequence, x, stream [B, D]; the caches' places move on in place, and so does the stream."""
        y, _, h, _ = efla.efla_rms_fwd(x, self.w_norm, stream, h=stream)
        xz = y @ self.w_in.t()
        u = efla.efla_conv_step(xz[..., : self.Di], self.w_conv, caches[0], self.b_conv, slots=slots)
        delta, B, C = self._inputs(u)
        o = efla.efla_scan_step(u, delta, -torch.exp(self.log_A), B, C, caches[1], self.skip, xz[..., self.Di:], self.b_dt, slots=slots)
        return o @ self.w_out.t(), h


def main():
    dev = torch.device("cuda:0")
    D, Di = 1024, 2048
    block = ScanBlock(D, Di, dev)
    gen = torch.Generator().manual_seed(1)

    # training: a few steps towards giving out the token before
    opt = torch.optim.Adam(block.parameters(), lr=1e-3)
    for it in range(20):
        x = torch.randn(4, 512, D, generator=gen).to(dev, torch.bfloat16)
        out, h = block.train_forward(x, torch.zeros_like(x))
        loss = F.mse_loss((h + out)[:, 1:].float(), x[:, :-1].float())
        opt.zero_grad()
        loss.backward()
        opt.step()
        if it % 5 == 4:
            print(f"step {it + 1}: loss {loss.item():.4f}")

    # serving: three prompts, their states at places 5, 0 and 3 of caches of 8, then eight tokens more
    lens = [300, 1, 77]
    offsets = torch.tensor([0, 300, 301, 378], dtype=torch.int32, device=dev)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device=dev)
    caches = block.caches(8)
    x = torch.randn(sum(lens), D, generator=gen).to(dev, torch.bfloat16)
    out, h = block.prefill(x, torch.zeros_like(x), offsets, caches, slots)
    last = (offsets[1:] - 1).long()
    token, stream = out[last], h[last]
    for _ in range(8):
        token, stream = block.decode(token, stream, caches, slots)
    efla.efla_get_status()
    print("served", len(lens), "sequences; |state|:", [f"{caches[1][s].norm().item():.2f}" for s in slots.tolist()])


if __name__ == "__main__":
    main()
