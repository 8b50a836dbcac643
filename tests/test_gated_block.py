"""The block that runs layer norm and the gated rule together: its gradients against the same block in
64 bits by autograd, and prompts then single tokens against the whole sequences at once."""
import math

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu


def plain_block(x, w_norm, b_norm, w_in, w_gate, b_gate, w_out, H, dk):
    """The block token by token, elementary operations."""
    B, L, D = x.shape
    m = x.mean(-1, keepdim=True)
    y = (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + 1e-5) * w_norm + b_norm
    p = y @ w_in.t()
    q, k, v = p[..., : 3 * H * dk].view(B, L, 3, H, dk).permute(2, 0, 3, 1, 4)
    q = q / math.sqrt(dk)
    beta = torch.sigmoid(p[..., 3 * H * dk:]).transpose(1, 2)
    g = -F.softplus(y @ w_gate.t() + b_gate).transpose(1, 2)
    lam = (k * k).sum(-1)
    alpha = -torch.expm1(-beta * lam) / lam
    S = x.new_zeros(B, H, dk, dk)
    o = []
    for t in range(L):
        S = S * torch.exp(g[:, :, t, None, None])
        r = v[:, :, t] - torch.einsum("bhij,bhi->bhj", S, k[:, :, t])
        S = S + torch.einsum("bhi,bhj->bhij", k[:, :, t] * alpha[:, :, t, None], r)
        o.append(torch.einsum("bhij,bhi->bhj", S, q[:, :, t]))
    return x + torch.stack(o, 1).reshape(B, L, H * dk) @ w_out.t()


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def test_training_gradients():
    """The block rounds to bf16 at its activations (a relative 2^-9 each, about ten in a row on any way
    through it): 5e-2 of a gradient's norm leaves room for their sum of squares and for the rule's memory."""
    from examples.gated_block import DK, GatedBlock
    dev = torch.device("cuda:0")
    block = GatedBlock(256, 2, dev, seed=3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(2, 150, 256, generator=gen).to(dev, torch.bfloat16)
    up = torch.randn(2, 150, 256, generator=gen).to(dev, torch.bfloat16)
    out = block.train_forward(x)
    grads = torch.autograd.grad(out, block.parameters(), up)
    ps = [t.detach().double().requires_grad_() for t in block.parameters()]
    ref = plain_block(x.double(), *ps, block.H, DK)
    want = torch.autograd.grad(ref, ps, up.double())
    assert rel(out, ref.detach()) < 2e-2
    for name, a, b in zip(("w_norm", "b_norm", "w_in", "w_gate", "b_gate", "w_out"), grads, want):
        assert rel(a, b) < 5e-2, name


def test_prompts_then_tokens():
    """States after prompts and single tokens are those of the whole sequences: both ways round q, k, v and the
    norm's output alike, so what differs is fp32 sums (2e-4 of the state); outputs differ by bf16's last bit."""
    import exact_flow_recurrence_gb300 as efla
    from examples.gated_block import DK, GatedBlock
    dev = torch.device("cuda:0")
    block = GatedBlock(512, 4, dev, seed=5)
    gen = torch.Generator().manual_seed(6)
    lens, more = [70, 1, 129], 5
    xs = [torch.randn(n + more, 512, generator=gen).to(dev, torch.bfloat16) for n in lens]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=dev)

    def offsets(ns):
        return torch.tensor([0] + ns, device=dev).cumsum(0).int()

    cache = torch.zeros(6, block.H, DK, DK, device=dev)
    block.prefill(torch.cat([x[:n] for x, n in zip(xs, lens)]), offsets(lens), cache, slots)
    outs = [block.decode(torch.stack([x[n + i] for x, n in zip(xs, lens)]), cache, slots) for i in range(more)]
    whole = torch.zeros_like(cache)
    ref = block.prefill(torch.cat(xs), offsets([n + more for n in lens]), whole, slots)
    efla.efla_get_status()
    end = 0
    for b, n in enumerate(lens):
        want = ref[end + n: end + n + more].double()
        got = torch.stack([o[b] for o in outs])
        assert rel(got, want) < 1e-2
        end += n + more
    assert rel(cache, whole.double()) < 2e-4
