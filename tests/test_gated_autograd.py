"""The example's differentiable forms of the norm and of the gated rule under autograd's own habits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _rule(seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = ((torch.randn(2, 2, 70, 128, generator=gen) / 8).bfloat16().cuda().requires_grad_() for _ in range(3))
    g = (-torch.rand(2, 2, 70, generator=gen)).cuda().requires_grad_()
    beta = torch.rand(2, 2, 70, generator=gen).cuda().requires_grad_()
    return [q, k, v, g, beta]


def _norm(seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(4, 6, 256, generator=gen).cuda().requires_grad_(), torch.rand(256, generator=gen).cuda().requires_grad_(),
            torch.rand(256, generator=gen).cuda().requires_grad_()]


def _cases():
    from examples.gated_block import GatedRule, LayerNorm
    return [(GatedRule, _rule()), (LayerNorm, _norm())]


@pytest.mark.parametrize("which", [0, 1])
def test_broadcast_gradients(which):
    """The gradient of a sum comes as one value with strides of zero, that of a sum over heads or rows as a
    broadcast row, a transposed loss's as columns: each gives what its dense copy gives."""
    fn, args = _cases()[which]
    out = fn.apply(*args)
    gen = torch.Generator().manual_seed(1)
    row = torch.randn(out.shape[-1], generator=gen).to(out.device, out.dtype)
    full = torch.randn(out.shape, generator=gen).to(out.device, out.dtype)
    for up in (torch.ones((), device=out.device, dtype=out.dtype).expand(out.shape), row.expand(out.shape),
               full.transpose(-1, -2).contiguous().transpose(-1, -2), full):
        got = torch.autograd.grad(out, args, up, retain_graph=True)
        want = torch.autograd.grad(out, args, up.clone(memory_format=torch.contiguous_format), retain_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    out.sum().backward()
    assert all(t.grad is not None for t in args)


@pytest.mark.parametrize("which", [0, 1])
def test_second_derivatives_are_refused(which):
    """The kernels' share of a second derivative is not there: autograd says so instead of leaving it out."""
    fn, args = _cases()[which]
    first = torch.autograd.grad(fn.apply(*args).float().square().sum(), args, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        sum(t.float().sum() for t in first).backward()
