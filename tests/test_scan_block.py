"""The block that runs RMS norm, convolution and selective scan together: its gradients against the same block in 64 bits
by autograd, prompts then single tokens against the whole sequences at once, and the 8-bit output of the norm in its place."""
import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu


def plain_block(x, stream, w_norm, w_in, w_conv, b_conv, w_x, w_dt, b_dt, log_A, skip, w_out, Di, R, N):
    """The block token by token, elementary operations."""
    h = x + stream
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5) * w_norm
    p = y @ w_in.t()
    u, z = p[..., :Di], p[..., Di:]
    taps = w_conv.shape[1]
    rows = F.pad(u, (0, 0, taps - 1, 0))
    u = b_conv + sum(rows[:, j: j + u.shape[1]] * w_conv[:, j] for j in range(taps))
    u = u * torch.sigmoid(u)
    q = u @ w_x.t()
    dt = F.softplus(q[..., :R] @ w_dt.t() + b_dt)
    B, C = q[..., R: R + N], q[..., R + N:]
    S, A, o = x.new_zeros(x.shape[0], Di, N), -torch.exp(log_A), []
    for t in range(x.shape[1]):
        S = torch.exp(dt[:, t, :, None] * A) * S + (dt[:, t] * u[:, t])[..., None] * B[:, t, None]
        o.append((S * C[:, t, None]).sum(-1))
    o = (torch.stack(o, 1) + skip * u) * z * torch.sigmoid(z)
    return o @ w_out.t(), h


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def make(D, Di, seed, *shape):
    from examples.scan_block import ScanBlock
    dev = torch.device("cuda:0")
    block = ScanBlock(D, Di, dev, seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    return block, [torch.randn(*shape, D, generator=gen).to(dev, torch.bfloat16) for _ in range(4)]


def test_training_gradients():
    """The block rounds to bf16 at its activations (a relative 2^-9 each, about ten in a row on any way through it): 5e-2 of a
    gradient's norm leaves room for their sum of squares and for the scan's memory.  h is rounded in the block, so is x + stream
    in the plain one's input."""
    from examples.scan_block import N
    block, (x, stream, up, down) = make(256, 384, 3, 2, 150)
    stream = ((x.float() + stream.float()).bfloat16().float() - x.float()).bfloat16()
    out, h = block.train_forward(x, stream)
    grads = torch.autograd.grad([out, h], block.parameters(), [up, down], allow_unused=True)
    ps = [t.detach().double().requires_grad_() for t in block.parameters()]
    ref, h_ref = plain_block(x.double(), stream.double(), *ps, block.Di, block.R, N)
    want = torch.autograd.grad(ref, ps, up.double())      # (h has no weight behind it)
    assert rel(out, ref.detach()) < 2e-2 and rel(h, h_ref.detach()) < 2 ** -8
    names = ("w_norm", "w_in", "w_conv", "b_conv", "w_x", "w_dt", "b_dt", "log_A", "skip", "w_out")
    for name, a, b in zip(names, grads, want):
        assert rel(a, b) < 5e-2, name


def test_gradients_of_the_stream():
    block, (x, stream, up, down) = make(256, 256, 5, 1, 70)
    x.requires_grad_()
    stream.requires_grad_()
    out, h = block.train_forward(x, stream)
    dx, ds = torch.autograd.grad([out, h], [x, stream], [up, down])
    assert torch.equal(dx, ds)
    out, h = block.train_forward(x, stream)
    dx, ds = torch.autograd.grad(h.sum(), [x, stream])     # (a gradient that comes broadcast, and none for the output)
    assert torch.equal(dx, torch.ones_like(dx)) and torch.equal(ds, dx)


def test_prompts_then_tokens():
    """States after prompts and single tokens are those of the whole sequences: both ways round the activations alike, so what
    differs is fp32 sums (2e-4 of the state); outputs differ by bf16's last bit."""
    import exact_flow_recurrence_gb300 as efla
    lens, more = [70, 1, 129, 2], 5
    block, (x, s, _, _) = make(512, 1024, 7, sum(lens) + len(lens) * more)
    dev = x.device
    xs, ss = x.split([n + more for n in lens]), s.split([n + more for n in lens])
    slots = torch.tensor([4, 0, 2, 5], dtype=torch.int32, device=dev)

    def offsets(ns):
        return torch.tensor([0] + ns, device=dev).cumsum(0).int()

    caches = block.caches(6)
    block.prefill(torch.cat([t[:n] for t, n in zip(xs, lens)]), torch.cat([t[:n] for t, n in zip(ss, lens)]), offsets(lens), caches, slots)
    outs = [block.decode(*(torch.stack([t[n + i] for t, n in zip(k, lens)]) for k in (xs, ss)), caches, slots) for i in range(more)]
    whole = block.caches(6)
    ref, h_ref = block.prefill(x, s, offsets([n + more for n in lens]), whole, slots)
    efla.efla_get_status()
    end = 0
    for b, n in enumerate(lens):
        at = slice(end + n, end + n + more)
        assert rel(torch.stack([o[b] for o, _ in outs]), ref[at].double()) < 1e-2
        assert torch.equal(torch.stack([h[b] for _, h in outs]), h_ref[at])
        end += n + more
    assert rel(caches[0], whole[0].double()) < 1e-2 and rel(caches[1], whole[1].double()) < 1e-2
    assert float(caches[1][[1, 3]].abs().max()) == 0.0


def test_decode_in_a_graph():
    """Tokens of a captured decode step, replayed on its own buffers, are those of the calls."""
    import exact_flow_recurrence_gb300 as efla
    block, (x, s, _, _) = make(256, 512, 9, 6)
    slots = torch.tensor([3, 1, 0, 2, 7, 5], dtype=torch.int32, device=x.device)
    caches, want = block.caches(8), block.caches(8)
    xi, si = x.clone(), s.clone()
    block.decode(xi, si.clone(), block.caches(8), slots)    # (libraries warm up outside the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h = block.decode(xi, si, caches, slots)
    for c in caches:
        c.zero_()
    for i in range(3):
        xi.copy_(x * (i + 1))
        si.copy_(s)
        graph.replay()
        ref, h_ref = block.decode(x * (i + 1), s.clone(), want, slots)
        efla.efla_get_status()
        assert torch.equal(out, ref) and torch.equal(h, h_ref)
    assert all(torch.equal(a, b) for a, b in zip(caches, want))


def test_8_bit_norm_feeds_the_projection():
    """y in 8 bits with its scales: each value is off by 2^-4 of itself at most, about 2^-5.5 at random, and a projection adds
    1024 of them at random signs: its norm moves by as much."""
    import exact_flow_recurrence_gb300 as efla
    block, (x, s, _, _) = make(1024, 512, 11, 33)
    y, _, h, _ = efla.efla_rms_fwd(x, block.w_norm, s)
    want = y.double() @ block.w_in.double().t()
    for group in (128, 1024):
        q, scale, h8, _ = efla.efla_rms_fwd(x, block.w_norm, s, group=group)
        efla.efla_get_status()
        got = (q.double().unflatten(-1, (-1, group)) * scale.double()[..., None]).flatten(-2) @ block.w_in.double().t()
        assert torch.equal(h8, h) and rel(got, want.detach()) < 2 ** -4.5


def test_example_runs(capsys):
    from examples import scan_block
    scan_block.main()
    assert "served 3 sequences" in capsys.readouterr().out
