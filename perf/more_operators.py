"""Measured cases of the short causal convolution, the selective scan and the residual's RMS norm.

Convolution (each channel by itself, W taps over the tokens up to its own):
    y_t = act(bias + sum_j w_j x_{t - (W - 1) + j}),   act the identity or x sigmoid(x)
Tokens before a sequence's first are its state's rows [W - 1, D], oldest first, or zeros.

Selective scan.  Channel d keeps N states and reads the B and C of group d // (D / G):
    dt = softplus(delta + delta_bias)                        (or delta + delta_bias itself)
    h <- e^{dt A} h + dt u B,   y = (sum_n C h + D u) z sigmoid(z)

RMS norm behind a residual's addition:
    h = x + residual (rounded to their type),   y = h rstd weight,   rstd = 1 / sqrt(mean(h^2) + eps)
with y in the type of x, or in e4m3 with a scale (largest |y| / 448) for 128 columns or for a row.

Operators: conv_fwd, conv_bwd, conv_step (one new token on a cache of states), scan_fwd, scan_bwd,
scan_step, rms_fwd, rms_bwd.
"""
import math

import torch

own = False
DEV = "cuda"
RANK = 64       # columns of a fused projection that lie in front of B and C (those that delta comes from)
TINY = 2.0 ** -126


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a training layer's scan: B8 L2048, 2048 channels of 16 states
        {"name": "scan_fwd_train", "op": "scan_fwd", "B": 8, "L": 2048, "D": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "packed": False, "state": False, "gate": True, "softplus": True},
        # prefill of 13 requests of different lengths packed on one axis, from and to states
        {"name": "scan_fwd_prefill_packed", "op": "scan_fwd", "B": 13, "L": 16384, "D": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "packed": True, "state": True, "gate": True, "softplus": True},
        # a short prompt in full precision, an odd width: latency
        {"name": "scan_fwd_short_f32", "op": "scan_fwd", "B": 1, "L": 77, "D": 200, "N": 8, "G": 2, "dtype": "f32",
         "packed": False, "state": True, "gate": False, "softplus": True},
        # gradients of a training layer: B4 L4096
        {"name": "scan_bwd_train", "op": "scan_bwd", "B": 4, "L": 4096, "D": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "packed": False, "state": False, "gate": True, "softplus": True},
        # gradients over packed sequences, two groups of wider states, states on both ends
        {"name": "scan_bwd_packed", "op": "scan_bwd", "B": 7, "L": 6001, "D": 1000, "N": 32, "G": 2, "dtype": "bf16",
         "packed": True, "state": True, "gate": False, "softplus": True},
        # a full batch decoding on a cache of states, in any order
        {"name": "scan_step_batch", "op": "scan_step", "B": 256, "D": 4096, "N": 16, "G": 1, "dtype": "bf16", "slots": True,
         "gate": True, "softplus": True},
        # the convolution in front of the training layer's scan
        {"name": "conv_fwd_train", "op": "conv_fwd", "B": 8, "L": 2048, "D": 2048, "W": 4, "dtype": "bf16", "packed": False,
         "state": False, "silu": True, "bias": True},
        # its gradients
        {"name": "conv_bwd_train", "op": "conv_bwd", "B": 4, "L": 4096, "D": 2048, "W": 4, "dtype": "bf16", "packed": False,
         "state": False, "silu": True, "bias": True},
        # one request decoding: the convolution of one token
        {"name": "conv_step_one", "op": "conv_step", "B": 1, "D": 2048, "W": 4, "dtype": "bf16", "slots": False, "silu": True,
         "bias": True},
        # the norm of a training batch, on the residual stream
        {"name": "rms_fwd_train", "op": "rms_fwd", "rows": 16384, "D": 2048, "dtype": "bf16", "wdtype": "f32", "residual": True,
         "quant": "none"},
        # the norm of a prompt whose next product reads 8 bits
        {"name": "rms_fwd_8bit", "op": "rms_fwd", "rows": 6001, "D": 2048, "dtype": "bf16", "wdtype": "f32", "residual": True,
         "quant": "group"},
        # its gradients on the training batch
        {"name": "rms_bwd_train", "op": "rms_bwd", "rows": 16384, "D": 2048, "dtype": "bf16", "wdtype": "f32", "residual": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd", "conv_step", "rms_fwd", "rms_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("rms"):
        d = _log(rng, 32, 8192)
        case = {"op": op, "rows": _log(rng, 1, min(65536, 16384 * 2048 // d)), "D": d, "dtype": dtype, "wdtype": rng.choice(["f32", "bf16"]),
                "residual": rng.random() < 0.7}
        return dict(case, quant=rng.choice(["none", "group", "row"])) if op == "rms_fwd" else case
    d = _log(rng, 32, 4096)
    if rng.random() < 0.7:
        d = -(-d // 8) * 8
    if op.startswith("conv"):
        case = {"op": op, "D": d, "W": rng.choice([4, 4, 3, 2]), "dtype": dtype, "silu": rng.random() < 0.7, "bias": rng.random() < 0.7}
        most = 16384 * 2048 // d
    else:
        n = rng.choice([16, 16, 16, 8, 32, 64, 4, 13])
        g = rng.choice([x for x in (1, 1, 1, 2, 4) if d % x == 0])
        case = {"op": op, "D": d, "N": n, "G": g, "dtype": dtype, "gate": rng.random() < 0.6, "softplus": rng.random() < 0.8}
        most = 16384 * 2048 * 16 // (d * n)
    if op.endswith("step"):
        return dict(case, B=_log(rng, 1, min(512, 256 * 4096 // d)), slots=rng.random() < 0.5)
    most = max(1, min(65536, most))
    packed = rng.random() < 0.4
    if packed:
        b = _log(rng, 1, min(32, most))
        length = _log(rng, b, min(16384, most))
    else:
        length = _log(rng, 1, min(16384, most))
        b = _log(rng, 1, max(1, min(64, most // length)))
    return dict(case, B=b, L=length, packed=packed, state=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lengths(case):
    """Where the packed sequences begin and end: unequal lengths that fill the axis."""
    import random
    r = random.Random(case["B"] * 1000003 + case["L"])
    cuts = sorted(r.randint(0, case["L"]) for _ in range(case["B"] - 1))
    return [0] + cuts + [case["L"]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s, dt = dict(case), _dtype(case["dtype"])
    d = case["D"]
    if case["op"].startswith("rms"):
        rows, w = case["rows"], _dtype(case["wdtype"])
        s["x"] = rnd(rows, d).to(dt)
        s["res"] = (3 * rnd(rows, d)).to(dt) if case["residual"] else None
        s["w"] = (1 + 0.2 * rnd(d)).to(w)
        s["eps"] = 1e-5
        if case["op"] == "rms_bwd":      # x is what the forward left: the stream h
            s["dy"] = rnd(rows, d).to(dt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + s["eps"])
        return s
    b = case["B"]
    step = case["op"].endswith("step")
    lead = (b,) if step else (case["L"],) if case["packed"] else (b, case["L"])
    fused = rnd(*lead, 2 * d).to(dt)     # x and its gate, as one projection writes them
    s["ends"] = _lengths(case) if not step and case["packed"] else None
    s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device=DEV) if s["ends"] else None
    places = b + b // 8 + 1 if step and case["slots"] else b
    if step:
        s["slots"] = torch.randperm(places, generator=gen, device=DEV)[:b].to(torch.int32) if case["slots"] else None
    if case["op"].startswith("conv"):
        w = case["W"]
        s["x"] = fused[..., :d]
        s["w"] = rnd(d, w) / math.sqrt(w)
        s["bias"] = 0.1 * rnd(d) if case["bias"] else None
        s["S"] = rnd(places, w - 1, d).to(dt) if step or case["state"] else None
        if case["op"] == "conv_bwd":
            s["dy"] = rnd(*lead, d).to(dt)
            s["dS"] = rnd(b, w - 1, d).to(dt) if case["state"] else None
        return s
    n, g = case["N"], case["G"]
    s["u"] = torch.nn.functional.silu(rnd(*lead, d)).to(dt)
    bc = rnd(*lead, RANK + 2 * g * n).to(dt)
    s["Bm"], s["C"] = (bc[..., RANK + i * g * n: RANK + (i + 1) * g * n].unflatten(-1, (g, n)) for i in (0, 1))
    s["A"] = -(1 + torch.arange(n, device=DEV)) * torch.exp(0.1 * rnd(d, n))
    # step sizes from 0.001 to 0.1, as such models begin with, spread by the input
    size = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(d, generator=gen, device=DEV))
    spread = 0.5 * rnd(*lead, d)
    if case["softplus"]:
        s["delta"], s["dbias"] = spread.to(dt), size + torch.log(-torch.expm1(-size))
    else:
        s["delta"], s["dbias"] = (size * torch.exp(spread)).to(dt), None
    s["skip"] = 1 + 0.1 * rnd(d)
    s["z"] = fused[..., d:] if case["gate"] else None
    s["S"] = 0.5 * rnd(places, d, n) if step or case["state"] else None
    if case["op"] == "scan_bwd":
        s["dy"] = rnd(*lead, d).to(dt)
        s["dS"] = 0.1 * rnd(b, d, n) if case["state"] else None
    return s


# ------------------------------------------------------------------------------ the plain form
def _flat(s, x):
    """[tokens, ...] of [B, L, ...], or of what is packed already."""
    return x if s["packed"] else x.flatten(0, 1)


def _ends(s):
    """The sequences' bounds on the axis of all tokens, each token's sequence and its place there."""
    ends = s["offsets"].long() if s["packed"] else torch.arange(s["B"] + 1, device=DEV) * s["L"]
    at = torch.arange(s["L"] if s["packed"] else s["B"] * s["L"], device=DEV)
    seq = torch.searchsorted(ends, at, right=True) - 1
    return ends, at, seq


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    sig = 1 / (1 + torch.exp(-x))
    return sig * (1 + x * (1 - sig))


def _dt(s, delta):
    x = delta if s["dbias"] is None else delta + s["dbias"]
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs())) if s["softplus"] else x


def _scan(a, w):
    """h_t = a_t h_{t-1} + w_t along dim 0 by doubling: after a step of `far`, (a, w) map the state 2 far tokens back."""
    far = 1
    while far < a.shape[0]:
        w[far:] += a[far:] * w[:-far]
        a[far:] = a[far:] * a[:-far]
        far *= 2
    return w


def _plain_scan(s):
    f, (ends, at, seq), dt = torch.float32, _ends(s), s["u"].dtype
    g, n = s["C"].shape[-2:]
    u, delta, bm, c = (_flat(s, s[k]).to(f) for k in ("u", "delta", "Bm", "C"))
    step = _dt(s, delta).unflatten(-1, (g, -1))
    u, bm, c, am = u.unflatten(-1, (g, -1)), bm[:, :, None], c[:, :, None], s["A"].unflatten(0, (g, -1))
    skip = s["skip"].unflatten(0, (g, -1))
    first, last = (at == ends[seq]), (at == ends[seq + 1] - 1)
    S0 = None if s["S"] is None else s["S"].unflatten(1, (g, -1))
    keep = torch.exp(step[..., None] * am)
    w = (step * u)[..., None] * bm
    if S0 is not None:
        w += torch.where(first[:, None, None, None], keep, 0.0) * S0[seq]
    h = _scan(torch.where(first[:, None, None, None], 0.0, keep), w)
    y = (h * c).sum(-1) + skip * u
    z = None if s["z"] is None else _flat(s, s["z"]).to(f).unflatten(-1, (g, -1))

    def tokens(x, of):
        return x.flatten(1, 2).to(dt).view(of.shape) if s["packed"] else x.flatten(1, 2).to(dt).unflatten(0, of.shape[:2])

    some = (ends[1:] > ends[:-1])[:, None, None]
    if s["op"] == "scan_fwd":
        y = tokens(y if z is None else y * _silu(z), s["u"])
        return (y,) if S0 is None else (y, torch.where(some, h[(ends[1:] - 1).clamp_min(0)].flatten(1, 2), s["S"]))
    dy = _flat(s, s["dy"]).to(f).unflatten(-1, (g, -1))
    gy = dy if z is None else dy * _silu(z)
    dc = (h * gy[..., None]).sum(2)
    h = torch.cat([torch.zeros_like(h[:1]), h[:-1]])     # the state that each token meets
    if S0 is None:
        h = torch.where(first[:, None, None, None], 0.0, h)
    else:
        h = torch.where(first[:, None, None, None], S0[seq], h)
    dS = None if s["dS"] is None else s["dS"].unflatten(1, (g, -1))
    p = c * gy[..., None]
    if dS is not None:
        p += torch.where(last[:, None, None, None], dS[seq], 0.0)
    after = torch.cat([keep[1:], torch.zeros_like(keep[:1])])
    after = torch.where(last[:, None, None, None], 0.0, after)
    p = _scan(after.flip(0), p.flip(0)).flip(0)
    del after
    s1 = (p * bm).sum(-1)
    db = (p * (step * u)[..., None]).sum(2)
    p *= keep
    dS0 = None if S0 is None else torch.where(some, p[ends[:-1].clamp_max(len(at) - 1)].flatten(1, 2), s["dS"])
    p *= h
    ddt = (p * am).sum(-1) + u * s1
    da = (p * step[..., None]).sum(0).flatten(0, 1)
    if s["softplus"]:
        x = delta if s["dbias"] is None else delta + s["dbias"]
        ddt = ddt / (1 + torch.exp(-x)).unflatten(-1, (g, -1))
    out = {"du": tokens(step * s1 + skip * gy, s["u"]), "ddelta": tokens(ddt, s["u"]), "dA": da,
           "dB": db.to(dt).view(s["Bm"].shape), "dC": dc.to(dt).view(s["C"].shape), "dD": (gy * u).sum(0).flatten()}
    if z is not None:
        out["dz"] = tokens(dy * y * _dsilu(z), s["u"])
    if s["dbias"] is not None:
        out["ddelta_bias"] = ddt.sum(0).flatten()
    if S0 is not None:
        out["dS0"] = dS0
    return out


def _plain_conv(s):
    f, (ends, at, seq), dt, wide = torch.float32, _ends(s), s["x"].dtype, s["W"] - 1
    x, num = _flat(s, s["x"]), torch.arange(s["B"], device=DEV)
    S0 = torch.zeros(s["B"], wide, x.shape[-1], dtype=dt, device=DEV) if s["S"] is None else s["S"]
    rows = torch.cat([S0.flatten(0, 1), x]).to(f)        # the states' rows, then the tokens
    old, back = s["B"] * wide, torch.arange(-wide, 1, device=DEV)

    def row(b, place):   # where the row at a place of sequence b lies (states' rows: places below 0)
        return torch.where(place >= 0, old + ends[b] + place, b * wide + wide + place)

    tap = row(seq[:, None], (at - ends[seq])[:, None] + back)
    pre = sum(rows[tap[:, j]] * s["w"][:, j] for j in range(s["W"]))
    pre = pre if s["bias"] is None else pre + s["bias"]
    if s["op"] == "conv_fwd":
        y = (_silu(pre) if s["silu"] else pre).to(dt).view(s["x"].shape)
        end = row(num[:, None], (ends[1:] - ends[:-1])[:, None] + back[:-1])
        return (y,) if s["S"] is None else (y, rows[end].to(dt))
    dy = _flat(s, s["dy"]).to(f)
    dp = dy * _dsilu(pre) if s["silu"] else dy
    # each row's sequence and place; tap j of the token at place + W - 1 - j reads it
    of = torch.cat([num.repeat_interleave(wide), seq])
    place = torch.cat([back[:-1].repeat(s["B"]), at - ends[seq]])
    length = (ends[1:] - ends[:-1])[of]
    users = place[:, None] - back
    inside = (users >= 0) & (users < length[:, None])
    users = torch.where(inside, ends[of][:, None] + users, 0)
    dr = sum(dp[users[:, j]] * s["w"][:, j] * inside[:, j, None] for j in range(s["W"]))
    if s["dS"] is not None:
        r = place - length + wide
        dr += s["dS"].to(f)[of, r.clamp_min(0)] * (r >= 0)[:, None]
    out = {"dx": dr[old:].to(dt).view(s["x"].shape), "dw": torch.stack([(dp * rows[tap[:, j]]).sum(0) for j in range(s["W"])], -1)}
    if s["bias"] is not None:
        out["dbias"] = dp.sum(0)
    if s["S"] is not None:
        out["dS0"] = dr[:old].view(s["S"].shape).to(dt)
    return out


def _plain_step(s):
    f, x = torch.float32, s["x" if s["op"] == "conv_step" else "u"]
    where = torch.arange(s["B"], device=DEV) if s["slots"] is None else s["slots"].long()
    if s["op"] == "conv_step":
        rows = torch.cat([s["S"][where], x[:, None]], 1)
        s["S"][where] = rows[:, 1:]
        y = (rows.to(f) * s["w"].t()).sum(1)
        y = y if s["bias"] is None else y + s["bias"]
        return (_silu(y) if s["silu"] else y).to(x.dtype), s["S"]
    rep = s["D"] // s["C"].shape[1]
    u, bm, c = x.to(f), s["Bm"].to(f).repeat_interleave(rep, 1), s["C"].to(f).repeat_interleave(rep, 1)
    step = _dt(s, s["delta"].to(f))
    h = torch.exp(step[..., None] * s["A"]) * s["S"][where] + (step * u)[..., None] * bm
    s["S"][where] = h
    y = (h * c).sum(-1) + s["skip"] * u
    return (y if s["z"] is None else y * _silu(s["z"].to(f))).to(x.dtype), s["S"]


def _plain_rms(s):
    f, x, w = torch.float32, s["x"], s["w"].float()
    if s["op"] == "rms_bwd":
        h, r = x.to(f), s["rstd"][:, None]
        p = s["dy"].to(f) * w
        dx = r * (p - h * (r * r * (p * h).mean(-1, keepdim=True)))
        dx = dx if s["res"] is None else dx + s["res"].to(f)
        return dx.to(x.dtype), (s["dy"].to(f) * h * r).sum(0).to(s["w"].dtype)
    h = x if s["res"] is None else (x.to(f) + s["res"].to(f)).to(x.dtype)
    v = h.to(f)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + s["eps"])
    y, stream = v * r * w, () if s["res"] is None else (h,)
    if s["quant"] == "none":
        return (y.to(x.dtype), r[:, 0]) + stream
    n = _group(s)
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % n)).unflatten(1, (-1, n))
    scale = y.abs().amax(-1).clamp_min(448 * TINY) / 448
    q = (y / scale[..., None]).clamp(-448, 448).flatten(1)[:, :x.shape[1]].to(torch.float8_e4m3fn)
    return (q, scale, r[:, 0]) + stream


def _group(s):
    return 128 if s["quant"] == "group" else s["D"]


# ------------------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if own:
        return _own(s)
    with torch.no_grad():
        return _plain_rms(s) if op.startswith("rms") else _plain_step(s) if op.endswith("step") else \
            _plain_conv(s) if op.startswith("conv") else _plain_scan(s)


def _own(s):
    import exact_flow_recurrence_gb300 as efla
    op = s["op"]
    if op == "rms_fwd":
        y, scale, h, rstd = efla.efla_rms_fwd(s["x"], s["w"], s["res"], eps=s["eps"], group=0 if s["quant"] == "none" else _group(s))
        return ((y,) if scale is None else (y, scale)) + (rstd,) + (() if s["res"] is None else (h,))
    if op == "rms_bwd":
        return efla.efla_rms_bwd(s["x"], s["w"], s["dy"], s["rstd"], dh=s["res"])
    if op == "conv_step":
        return efla.efla_conv_step(s["x"], s["w"], s["S"], s["bias"], slots=s["slots"], silu=s["silu"]), s["S"]
    if op == "conv_fwd":
        y, last = efla.efla_conv_fwd(s["x"], s["w"], s["bias"], s["S"], offsets=s["offsets"], silu=s["silu"],
                                     want_state=s["S"] is not None)
        return (y,) if last is None else (y, last)
    if op == "conv_bwd":
        d = efla.efla_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["S"], s["dS"], offsets=s["offsets"], silu=s["silu"],
                               want_dS0=s["S"] is not None)
        return {k: v for k, v in zip(("dx", "dw", "dbias", "dS0"), d) if v is not None}
    scan = (s["u"], s["delta"], s["A"], s["Bm"], s["C"])
    if op == "scan_step":
        return efla.efla_scan_step(*scan, s["S"], s["skip"], s["z"], s["dbias"], slots=s["slots"], softplus=s["softplus"]), s["S"]
    if op == "scan_fwd":
        y, last = efla.efla_scan_fwd(*scan, s["skip"], s["z"], s["dbias"], s["S"], offsets=s["offsets"], softplus=s["softplus"],
                                     want_state=s["S"] is not None)
        return (y,) if last is None else (y, last)
    d = efla.efla_scan_bwd(*scan, s["dy"], s["skip"], s["z"], s["dbias"], s["S"], s["dS"], offsets=s["offsets"],
                           softplus=s["softplus"], want_dS0=s["S"] is not None)
    return {k: v for k, v in zip(("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dS0"), d) if v is not None}


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e, d, op = 2 if case["dtype"] == "bf16" else 4, case["D"], case["op"]
    if op.startswith("rms"):
        n, we = case["rows"] * d, d * (2 if case["wdtype"] == "bf16" else 4)
        if op == "rms_bwd":
            return {"bytes": n * e * (4 if case["residual"] else 3) + case["rows"] * 4 + 2 * we, "flops": 9 * n}
        groups = 0 if case["quant"] == "none" else -(-d // _group(case)) * case["rows"]
        out = n * e if case["quant"] == "none" else n + 4 * groups
        return {"bytes": n * e * (3 if case["residual"] else 1) + out + case["rows"] * 4 + we, "flops": 5 * n}
    step = op.endswith("step")
    rows = case["B"] if step else case["L"] * (1 if case["packed"] else case["B"])
    n, seqs = rows * d, case["B"]
    if op.startswith("conv"):
        w = case["W"]
        state = seqs * (w - 1) * d * e if step or case["state"] else 0
        par = d * 4 * (w + (1 if case["bias"] else 0))
        if op == "conv_bwd":
            return {"bytes": 3 * n * e + 3 * state + 2 * par, "flops": n * (6 * w + (8 if case["silu"] else 0))}
        return {"bytes": 2 * n * e + 2 * state + par, "flops": n * (2 * w + (4 if case["silu"] else 0))}
    m, gate = case["N"], 1 if case["gate"] else 0
    state = seqs * d * m * 4 if step or case["state"] else 0
    bc, par = 2 * rows * case["G"] * m * e, d * (m + 2) * 4
    # a state's update and read: the decay's exponent and power, its product, the input's, the output's
    if op == "scan_bwd":
        return {"bytes": (5 + 2 * gate) * n * e + 2 * bc + 2 * par + 3 * state, "flops": 23 * n * m}
    return {"bytes": (3 + gate) * n * e + bc + par + 2 * state, "flops": 8 * n * m}


# ------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"].startswith("rms"):
            return _exact_rms(s)
        return _exact_conv(s) if case["op"].startswith("conv") else _exact_scan(s)


def _exact_rms(s):
    w = s["w"].double()
    if s["op"] == "rms_bwd":
        h, r, dy = s["x"].double(), s["rstd"].double(), s["dy"].double()
        g = torch.einsum("rd,d->rd", dy, w)
        dx = g * r[:, None] - h * (torch.einsum("rd,rd->r", g, h) * r ** 3 / h.shape[1])[:, None]
        return (dx if s["res"] is None else dx + s["res"].double()), torch.einsum("rd,rd,r->d", dy, h, r)
    h = s["x"].double() if s["res"] is None else (s["x"].double() + s["res"].double()).to(s["x"].dtype).double()
    r = (h.pow(2).sum(-1) / h.shape[1] + s["eps"]).rsqrt()
    y = torch.einsum("rd,r,d->rd", h, r, w)
    stream = () if s["res"] is None else (h,)
    if s["quant"] == "none":
        return (y, r) + stream
    parts = [p.abs().max(1).values.clamp_min(448 * TINY) / 448 for p in y.split(_group(s), 1)]
    scale = torch.stack(parts, 1)
    return (torch.cat([p / m[:, None] for p, m in zip(y.split(_group(s), 1), parts)], 1), scale, r) + stream


def _sequences(s, names):
    """Each sequence's tokens of the named inputs, in 64 bits, as [1, length, ...] (or the whole batch at once)."""
    if s["op"].endswith("step"):
        return [(slice(None), {k: s[k].double()[:, None] for k in names if s.get(k) is not None})]
    if not s["packed"]:
        return [(slice(None), {k: s[k].double() for k in names if s.get(k) is not None})]
    return [(slice(b, b + 1), {k: s[k][lo:hi].double()[None] for k in names if s.get(k) is not None})
            for b, (lo, hi) in enumerate(zip(s["ends"], s["ends"][1:]))]


def _whole(s, parts):
    """The sequences' results as one call lays them out."""
    return parts[0] if not s.get("packed") else torch.cat(parts, 1)[0]


def _cache(s):
    return torch.arange(s["B"], device=DEV) if s["slots"] is None else s["slots"].long()


def _exact_conv(s):
    w, wide = s["w"].double(), s["W"] - 1
    step = s["op"] == "conv_step"
    start = None if s["S"] is None else s["S"].double()[_cache(s)] if step else s["S"].double()
    ys, last, grads = [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(w[:, 0])
    for at, t in _sequences(s, ("x", "dy")):
        x = t["x"]
        length = x.shape[1]
        old = x.new_zeros(x.shape[0], wide, x.shape[2]) if start is None else start[at]
        both = torch.cat([old, x], 1)
        win = both.unfold(1, wide + 1, 1) if length else x.new_zeros(x.shape[0], 0, x.shape[2], wide + 1)   # [b, length, d, W]
        pre = torch.einsum("bldw,dw->bld", win, w) + (0 if s["bias"] is None else s["bias"].double())
        sig = torch.sigmoid(pre)
        if s["op"] != "conv_bwd":
            ys.append(pre * sig if s["silu"] else pre)
            last.append(both[:, length:])
            continue
        dp = t["dy"] * (sig * (1 + pre * (1 - sig)) if s["silu"] else 1)
        dw += torch.einsum("bld,bldw->dw", dp, win)
        db += dp.sum((0, 1))
        dr = torch.zeros_like(both)
        for j in range(wide + 1):
            dr[:, j:j + length] += dp * w[:, j]
        if s["dS"] is not None:
            dr[:, length:] += s["dS"].double()[at]
        ys.append(dr[:, wide:])
        last.append(dr[:, :wide])
    if step:
        cache = s["S"].double()
        cache[_cache(s)] = last[0]
        return ys[0][:, 0], cache
    if s["op"] == "conv_fwd":
        return (_whole(s, ys),) if s["S"] is None else (_whole(s, ys), torch.cat(last))
    out = {"dx": _whole(s, ys), "dw": dw}
    if s["bias"] is not None:
        out["dbias"] = db
    if s["S"] is not None:
        out["dS0"] = torch.cat(last)
    return out


def _exact_scan(s):
    """Token by token, every sequence of a batch at once; the gradients walk back over the states kept."""
    A, D, n = s["A"].double(), s["skip"].double(), s["N"]
    step, rep = s["op"] == "scan_step", s["D"] // s["G"]
    start = None if s["S"] is None else s["S"].double()[_cache(s)] if step else s["S"].double()
    parts, last = {}, []
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(D), torch.zeros_like(D)

    def wide(x):    # a group's values for each of its channels
        return x.repeat_interleave(rep, 1)

    for at, t in _sequences(s, ("u", "delta", "Bm", "C", "z", "dy")):
        u = t["u"]
        raw = t["delta"] + (0 if s["dbias"] is None else s["dbias"].double())
        dt = torch.nn.functional.softplus(raw, threshold=60) if s["softplus"] else raw
        h = u.new_zeros(u.shape[0], s["D"], n) if start is None else start[at]
        kept, y = [], torch.empty_like(u)
        for i in range(u.shape[1]):
            if s["op"] == "scan_bwd":
                kept.append(h)
            h = torch.exp(dt[:, i, :, None] * A) * h + (dt[:, i] * u[:, i])[..., None] * wide(t["Bm"][:, i])
            y[:, i] = torch.einsum("bdn,bdn->bd", h, wide(t["C"][:, i]))
        y += D * u
        gate = torch.ones_like(u)
        if s["z"] is not None:
            sig = torch.sigmoid(t["z"])
            gate = t["z"] * sig
        if s["op"] != "scan_bwd":
            parts.setdefault("y", []).append(y * gate)
            last.append(h)
            continue
        gy = t["dy"] * gate
        r = {"du": D * gy, "ddelta": torch.zeros_like(u), "dB": torch.zeros_like(t["Bm"]), "dC": torch.zeros_like(t["C"])}
        if s["z"] is not None:
            r["dz"] = t["dy"] * y * (sig + gate * (1 - sig))
        p = torch.zeros_like(h) if s["dS"] is None else s["dS"].double()[at]
        for i in range(u.shape[1] - 1, -1, -1):
            keep = torch.exp(dt[:, i, :, None] * A)
            bm = wide(t["Bm"][:, i])
            new = keep * kept[i] + (dt[:, i] * u[:, i])[..., None] * bm
            r["dC"][:, i] = (new * gy[:, i, :, None]).unflatten(1, (-1, rep)).sum(2)
            p = p + gy[:, i, :, None] * wide(t["C"][:, i])
            r["dB"][:, i] = (p * (dt[:, i] * u[:, i])[..., None]).unflatten(1, (-1, rep)).sum(2)
            b = torch.einsum("bdn,bdn->bd", p, bm)
            r["du"][:, i] += dt[:, i] * b
            p = p * keep
            e = p * kept[i]
            r["ddelta"][:, i] = torch.einsum("bdn,dn->bd", e, A) + u[:, i] * b
            dA += torch.einsum("bdn,bd->dn", e, dt[:, i])
            kept[i] = None
        if s["softplus"]:
            r["ddelta"] *= torch.sigmoid(raw)
        dD += torch.einsum("bld,bld->d", gy, u)
        dbias += r["ddelta"].sum((0, 1))
        for k, v in r.items():
            parts.setdefault(k, []).append(v)
        last.append(p)
    if step:
        cache = s["S"].double()
        cache[_cache(s)] = last[0]
        return parts["y"][0][:, 0], cache
    whole = {k: _whole(s, v) for k, v in parts.items()}
    if s["op"] == "scan_fwd":
        return (whole["y"],) if s["S"] is None else (whole["y"], torch.cat(last))
    out = dict(whole, dA=dA, dD=dD)
    if s["dbias"] is not None:
        out["ddelta_bias"] = dbias
    if s["S"] is not None:
        out["dS0"] = torch.cat(last)
    return out
