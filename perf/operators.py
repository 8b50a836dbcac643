"""Measured cases of the gated delta rule and of layer norm.

The gated delta rule keeps, for each sequence and head, a state S [dk, dv] and for each token
    S <- e^{g_t} S
    S <- S + alpha_t k_t (v_t - S^T k_t)^T,     o_t = S^T q_t
with g_t <= 0 the log of the token's decay, and alpha_t = beta_t ("euler", the delta rule) or
alpha_t = (1 - e^{-beta_t ||k_t||^2}) / ||k_t||^2 ("exact", the exact flow of the key direction).
Value head h reads the query and key of head h // (H / Hk).

Operators: gated_fwd (a whole sequence, chunked), gated_bwd (its gradients), gated_step (one new
token on a cache of states), norm_fwd and norm_bwd (layer norm over the last dimension).
"""
import math

import torch

own = False
DEV = "cuda"
C = 64          # tokens a chunk of the plain form


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a training layer of the 340M-parameter shape: B8 H8 L2048, no state carried
        {"name": "fwd_train", "op": "gated_fwd", "B": 8, "H": 8, "Hk": 8, "L": 2048, "dk": 128, "dv": 128,
         "dtype": "bf16", "packed": False, "token_first": False, "state": False, "mode": "euler"},
        # prefill of requests of different lengths packed on one axis, two value heads to a key
        # head, token-major as a projection writes them, from and to the state cache
        {"name": "fwd_prefill_packed", "op": "gated_fwd", "B": 13, "H": 16, "Hk": 8, "L": 16384, "dk": 128,
         "dv": 128, "dtype": "bf16", "packed": True, "token_first": True, "state": True, "mode": "euler"},
        # one long document: few heads, a long chain
        {"name": "fwd_long", "op": "gated_fwd", "B": 1, "H": 16, "Hk": 16, "L": 16384, "dk": 128, "dv": 128,
         "dtype": "bf16", "packed": False, "token_first": False, "state": True, "mode": "exact"},
        # a short prompt in full precision: latency
        {"name": "fwd_short_f32", "op": "gated_fwd", "B": 1, "H": 4, "Hk": 2, "L": 77, "dk": 64, "dv": 48,
         "dtype": "f32", "packed": False, "token_first": True, "state": True, "mode": "euler"},
        # gradients of a training layer of the 1.3B-parameter shape: B4 H16 L4096
        {"name": "bwd_train", "op": "gated_bwd", "B": 4, "H": 16, "Hk": 16, "L": 4096, "dk": 128, "dv": 128,
         "dtype": "bf16", "packed": False, "token_first": False, "state": False, "mode": "euler"},
        # gradients over packed sequences, shared key heads, narrower values, states on both ends
        {"name": "bwd_packed", "op": "gated_bwd", "B": 7, "H": 8, "Hk": 4, "L": 6001, "dk": 128, "dv": 64,
         "dtype": "bf16", "packed": True, "token_first": True, "state": True, "mode": "exact"},
        # one request decoding
        {"name": "step_one", "op": "gated_step", "B": 1, "H": 16, "Hk": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "slots": False, "mode": "euler"},
        # a full batch decoding on a cache of states, in any order
        {"name": "step_batch", "op": "gated_step", "B": 256, "H": 16, "Hk": 8, "dk": 128, "dv": 128,
         "dtype": "bf16", "slots": True, "mode": "euler"},
        # the norm before a decode step of a few requests
        {"name": "norm_fwd_decode", "op": "norm_fwd", "rows": 4, "D": 1024, "dtype": "bf16", "wdtype": "f32", "bias": True},
        # the norm of a training batch, 1.3B-parameter width
        {"name": "norm_fwd_train", "op": "norm_fwd", "rows": 16384, "D": 2048, "dtype": "bf16", "wdtype": "f32", "bias": True},
        # a ragged batch of an odd width in full precision
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 1001, "D": 999, "dtype": "f32", "wdtype": "f32", "bias": True},
        # its gradients on the training batch
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 16384, "D": 2048, "dtype": "bf16", "wdtype": "f32", "bias": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "gated_step", "norm_fwd", "norm_bwd"])
    if op.startswith("norm"):
        d = _log(rng, 32, 8192)
        return {"op": op, "rows": _log(rng, 1, min(65536, (16384 * 2048) // d)), "D": d, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "wdtype": rng.choice(["f32", "bf16"]), "bias": rng.random() < 0.7}
    hk = _log(rng, 1, 16)
    h = hk * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([128, 128, 64, 96, 48]), rng.choice([128, 128, 64, 80, 32])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    mode = rng.choice(["euler", "euler", "exact"])
    if op == "gated_step":
        return {"op": op, "B": _log(rng, 1, 4096 // h), "H": h, "Hk": hk, "dk": dk, "dv": dv, "dtype": dtype,
                "slots": rng.random() < 0.5, "mode": mode}
    tokens = (262144 if dtype == "bf16" else 16384) // h      # B L at most
    packed = rng.random() < 0.4
    if packed:
        b = _log(rng, 1, 32)
        length = _log(rng, b, min(16384, tokens))
    else:
        length = _log(rng, 1, min(16384, tokens))
        b = _log(rng, 1, max(1, min(64, tokens // length)))
    return {"op": op, "B": b, "H": h, "Hk": hk, "L": length, "dk": dk, "dv": dv, "dtype": dtype, "packed": packed,
            "token_first": rng.random() < 0.5, "state": rng.random() < 0.6, "mode": mode}


def _lengths(case):
    """Lengths of a packed case's B sequences, L tokens in all: uneven, some of them empty."""
    b, total = case["B"], case["L"]
    w = [((i * 2654435761 + total * 40503) % 1009) ** 2 * (i % 5 != 3) for i in range(b)]
    w[-1] += 1
    ends = [0]
    for i in range(b):
        ends.append(total * sum(w[:i + 1]) // sum(w))
    return ends


_T = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = {"case": case, "op": case["op"]}
    dt = _T[case["dtype"]]
    if case["op"].startswith("norm"):
        r, d = case["rows"], case["D"]
        s["x"] = (rnd(r, d) * (1 + rnd(r, 1).abs()) + 0.5 * rnd(r, 1)).to(dt)
        s["w"] = (1 + 0.1 * rnd(d)).to(_T[case["wdtype"]])
        s["b"] = (0.1 * rnd(d)).to(_T[case["wdtype"]]) if case["bias"] else None
        s["eps"] = 1e-5
        if case["op"] == "norm_bwd":
            x = s["x"].float()      # what the forward pass kept of each row: its mean and 1 / deviation
            mean = x.mean(-1)
            s["stats"] = torch.stack([mean, torch.rsqrt((x - mean[:, None]).square().mean(-1) + s["eps"])], -1)
            s["dy"] = rnd(r, d).to(dt)
        return s
    b, h, hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    length = case.get("L", 1)
    rows = 1 if case.get("packed") else b
    first = case.get("token_first")

    def tokens(heads, d):           # [rows, heads, length, d], stored head-major or token-major
        return rnd(rows, length, heads, d).transpose(1, 2) if first else rnd(rows, heads, length, d)

    def as_is(x):                   # the type of the tokens, in the same order of storage
        return x.to(dt)

    def scalar():
        return rnd(rows, length, h).transpose(1, 2) if first else rnd(rows, h, length)

    k = tokens(hk, dk)
    k = k / k.norm(dim=-1, keepdim=True)
    if case["mode"] == "exact":     # keys of different norms are what the exact flow is for
        k = k * torch.exp(0.5 * rnd(rows, hk, length, 1))
    rate = torch.exp(math.log(0.01) + (math.log(1.0) - math.log(0.01)) * torch.rand(h, generator=gen, device=DEV))
    s["q"], s["k"], s["v"] = as_is(tokens(hk, dk) / math.sqrt(dk)), as_is(k), as_is(tokens(h, dv))
    s["g"] = -rate[None, :, None] * torch.nn.functional.softplus(scalar())
    s["beta"] = torch.sigmoid(scalar())
    s["mode"] = case["mode"]
    if case["op"] == "gated_step":
        for n in ("q", "k", "v", "g", "beta"):
            s[n] = s[n][:, :, 0].contiguous()
        n = b + b // 8 + 1 if case["slots"] else b
        s["S"] = 0.2 * rnd(n, h, dk, dv)
        s["slots"] = torch.randperm(n, generator=gen, device=DEV)[:b].to(torch.int32) if case["slots"] else None
        return s
    s["ends"] = _lengths(case) if case["packed"] else None
    s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device=DEV) if case["packed"] else None
    s["S0"] = 0.2 * rnd(b, h, dk, dv) if case["state"] else None
    if case["op"] == "gated_bwd":
        s["dO"] = as_is(tokens(h, dv))
        s["dS"] = 0.1 * rnd(b, h, dk, dv) if case["state"] else None
    if case["packed"]:              # one axis of tokens: [heads, tokens, d]
        for n in ("q", "k", "v", "g", "beta", "dO"):
            if n in s:
                s[n] = s[n][0]
        longest = max(e - a for a, e in zip(s["ends"], s["ends"][1:]))
        at = torch.tensor(s["ends"][:-1], device=DEV)[:, None] + torch.arange(longest, device=DEV)
        s["at"], s["live"] = at.clamp_max(length - 1), at < torch.tensor(s["ends"][1:], device=DEV)[:, None]
    return s


# ------------------------------------------------------------------------------ plain forms
def _alpha(k, beta, mode):
    if mode == "euler":
        return beta
    lam = (k * k).sum(-1)
    safe = torch.where(lam > 0, lam, 1.0)
    return torch.where(lam > 0, -torch.expm1(-beta * lam) / safe, beta)


def _inverse(a):
    """(I + A)^{-1} of strictly lower triangular matrices [..., C, C], by doubling its diagonal blocks."""
    t = torch.ones(*a.shape[:-2], C, 1, 1, dtype=a.dtype, device=a.device)
    w = 1
    while w < C:
        n = C // w
        i = torch.arange(0, n, 2, device=a.device)
        below = a.unflatten(-1, (n, w)).unflatten(-3, (n, w)).transpose(-3, -2)[..., i + 1, i, :, :]
        top, low = t[..., 0::2, :, :], t[..., 1::2, :, :]
        t = torch.cat([torch.cat([top, torch.zeros_like(top)], -1), torch.cat([-(low @ below @ top), low], -1)], -2)
        w *= 2
    return t[..., 0, :, :]


def _plain_fwd(q, k, v, g, beta, state, mode):
    """[B, H, L, d] in 32 bits, L tokens in chunks of C; returns o and the last state."""
    b, h, length, dv = v.shape
    k, q = (x.repeat_interleave(h // x.shape[1], 1) for x in (k, q))
    alpha = _alpha(k, beta, mode)
    n = -(-length // C)
    pad = n * C - length

    def chunks(x):
        if pad:
            x = torch.cat([x, torch.zeros(*x.shape[:2], pad, *x.shape[3:], dtype=x.dtype, device=x.device)], 2)
        return x.unflatten(2, (n, C))

    q, k, v, g, alpha = (chunks(x) for x in (q, k, v, g, alpha))
    c = g.cumsum(-1)
    i = torch.arange(C, device=c.device)
    decay = torch.where(i[:, None] >= i, c[..., :, None] - c[..., None, :], -torch.inf).exp()
    t = _inverse(torch.where(i[:, None] > i, alpha[..., None] * (k @ k.mT) * decay, 0.0))
    p = (q @ k.mT) * decay
    up, last = c.exp()[..., None], c[..., -1:, None]
    rest = (c[..., -1:] - c).exp()[..., None]
    state = torch.zeros(b, h, k.shape[-1], dv, device=v.device) if state is None else state
    out = []
    for j in range(n):
        u = t[:, :, j] @ (alpha[:, :, j, :, None] * (v[:, :, j] - up[:, :, j] * (k[:, :, j] @ state)))
        out.append(up[:, :, j] * (q[:, :, j] @ state) + p[:, :, j] @ u)
        state = last[:, :, j].exp() * state + (rest[:, :, j] * k[:, :, j]).mT @ u
    return torch.cat(out, 2)[:, :, :length], state


def _spread(s, x):
    """Packed [heads, T, ...] as one padded row a sequence, [B, heads, longest, ...]; zeros where it has no token."""
    y = x[:, s["at"]].transpose(0, 1)
    live = s["live"][:, None]
    return torch.where(live[..., None] if x.dim() == 3 else live, y, 0.0)


def _gather(s, y):
    """The tokens of padded rows, back on one axis."""
    return y.transpose(1, 2)[s["live"]].transpose(0, 1)


def _rows(s, names, kind=torch.float32):
    x = [s[n].to(kind) for n in names]
    return [_spread(s, y) for y in x] if s["ends"] else x


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(-1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + s["eps"])
        y = (x - mean) * rstd * s["w"].float()
        y = y if s["b"] is None else y + s["b"].float()
        return y.to(s["x"].dtype), torch.cat([mean, rstd], -1)
    if op == "norm_bwd":
        dy, stats = s["dy"].float(), s["stats"]
        rstd = stats[:, 1:]
        xh = (s["x"].float() - stats[:, :1]) * rstd
        d = dy * s["w"].float()
        dx = rstd * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
        dw = (dy * xh).sum(0).to(s["w"].dtype)
        return (dx.to(s["x"].dtype), dw) + (() if s["b"] is None else (dy.sum(0).to(s["w"].dtype),))
    if op == "gated_step":
        r = s["v"].shape[1] // s["k"].shape[1]
        q, k, v = s["q"].float().repeat_interleave(r, 1), s["k"].float().repeat_interleave(r, 1), s["v"].float()
        slots = None if s["slots"] is None else s["slots"].long()
        state = (s["S"] if slots is None else s["S"][slots]) * s["g"].exp()[..., None, None]
        err = v - (state * k[..., None]).sum(-2)
        state = state + (_alpha(k, s["beta"], s["mode"])[..., None] * k)[..., None] * err[..., None, :]
        if slots is None:
            s["S"].copy_(state)
        else:
            s["S"][slots] = state
        return (state * q[..., None]).sum(-2).to(s["v"].dtype), s["S"]
    dt = s["v"].dtype
    if op == "gated_fwd":
        o, state = _plain_fwd(*_rows(s, ("q", "k", "v", "g", "beta")), s["S0"], s["mode"])
        o = (_gather(s, o) if s["ends"] else o).to(dt)
        return (o, state) if s["S0"] is not None else (o,)
    with torch.enable_grad():
        names = ("q", "k", "v", "g", "beta") + (("S0",) if s["S0"] is not None else ())
        leaf = [s[n].detach().float().requires_grad_() for n in names]
        x = [_spread(s, y) for y in leaf[:5]] if s["ends"] else leaf[:5]
        o, state = _plain_fwd(*x, leaf[5] if len(leaf) > 5 else None, s["mode"])
        o = _gather(s, o) if s["ends"] else o
        outs, grads = ([o], [s["dO"].float()]) if s["dS"] is None else ([o, state], [s["dO"].float(), s["dS"]])
        d = torch.autograd.grad(outs, leaf, grads)
    return tuple(x.to(dt) for x in d[:3]) + tuple(d[3:])


def run(state):
    if not own:
        with torch.no_grad():
            return _plain(state)
    import exact_flow_recurrence_gb300 as efla
    s, op = state, state["op"]
    if op == "norm_fwd":
        return efla.efla_norm_fwd(s["x"], s["w"], s["b"], eps=s["eps"])
    if op == "norm_bwd":
        dx, dw, db = efla.efla_norm_bwd(s["x"], s["w"], s["dy"], s["stats"], want_bias=s["b"] is not None)
        return (dx, dw) if db is None else (dx, dw, db)
    mode = efla.EXACT if s["mode"] == "exact" else efla.EULER
    if op == "gated_step":
        return efla.efla_gated_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], slots=s["slots"], mode=mode), s["S"]
    if op == "gated_fwd":
        o, last = efla.efla_gated_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], offsets=s["offsets"], mode=mode,
                                      want_state=s["S0"] is not None)
        return (o, last) if last is not None else (o,)
    d = efla.efla_gated_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dO"], s["S0"], s["dS"], offsets=s["offsets"], mode=mode,
                            want_dS0=s["S0"] is not None)
    return tuple(d if d[5] is not None else d[:5])


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"].startswith("norm"):
        n, e, w = case["rows"] * case["D"], 2 if case["dtype"] == "bf16" else 4, 2 if case["wdtype"] == "bf16" else 4
        two = 2 if case["bias"] else 1
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * e + two * case["D"] * w + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + (1 + two) * case["D"] * w + 8 * case["rows"], "flops": 14 * n}
    b, h, hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    e = 2 if case["dtype"] == "bf16" else 4
    seqs = b
    toks = case["B"] if case["op"] == "gated_step" else case["L"] * (1 if case["packed"] else b)
    qk, v, gates, states = toks * hk * dk * e, toks * h * dv * e, toks * h * 4, seqs * h * dk * dv * 4
    step = 6 * dk * dv * toks * h            # S^T k, the rank-one update, S^T q
    if case["op"] == "gated_step":
        return {"bytes": 2 * qk + 2 * v + 2 * gates + 2 * states, "flops": step}
    carried = states if case["state"] else 0
    if case["op"] == "gated_fwd":
        return {"bytes": 2 * qk + 2 * v + 2 * gates + 2 * carried, "flops": step}
    return {"bytes": 4 * qk + 3 * v + 4 * gates + 3 * carried, "flops": 3 * step}


# ------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact_norm(s) if s["op"].startswith("norm") else _exact_gated(s)


def _exact_norm(s):
    x, w = s["x"].double(), s["w"].double()
    if s["op"] == "norm_fwd":
        mean = x.mean(-1)
        rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(-1) + s["eps"])
        y = (x - mean[:, None]) * rstd[:, None] * w
        return y if s["b"] is None else y + s["b"].double(), torch.stack([mean, rstd], -1)
    dy, mean, rstd = s["dy"].double(), s["stats"][:, 0].double(), s["stats"][:, 1].double()
    d, n = x.shape[1], x - mean[:, None]
    wd = w * dy
    dx = rstd[:, None] * (wd - wd.sum(-1, keepdim=True) / d - n * (rstd ** 2 * (wd * n).sum(-1) / d)[:, None])
    dw = torch.einsum("rd,rd,r->d", dy, n, rstd)
    return (dx, dw) if s["b"] is None else (dx, dw, dy.sum(0))


def _exact_gated(s):
    """Token by token, every sequence at once; the gradients walk back over recomputed states."""
    if s["op"] == "gated_step":
        q, k, v, g, beta = (s[n].double().unsqueeze(2) for n in ("q", "k", "v", "g", "beta"))
    else:
        q, k, v, g, beta = _rows(s, ("q", "k", "v", "g", "beta"), torch.float64)
    b, h, length, dv = v.shape
    rep = h // k.shape[1]
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    lam = (k ** 2).sum(-1)
    if s["mode"] == "exact":
        alpha = torch.where(lam > 0, -torch.expm1(-beta * lam) / lam.clamp_min(1e-300), beta)
    else:
        alpha = beta
    f = g.exp()

    def token(state, t):
        state = state * f[:, :, t, None, None]
        r = v[:, :, t] - torch.einsum("bhkv,bhk->bhv", state, k[:, :, t])
        return state, r, state + (alpha[:, :, t, None] * k[:, :, t])[..., None] * r[..., None, :]

    if s["op"] == "gated_step":
        where = torch.arange(b, device=DEV) if s["slots"] is None else s["slots"].long()
        cache = s["S"].double()
        new = token(cache[where], 0)[2]
        cache[where] = new
        return torch.einsum("bhkv,bhk->bhv", new, q[:, :, 0]), cache
    state = torch.zeros(b, h, k.shape[-1], dv, dtype=torch.float64, device=DEV) if s["S0"] is None else s["S0"].double()
    marks, o, seg = {}, torch.empty_like(v), 32
    for t in range(length):
        if t % seg == 0:
            marks[t] = state
        state = token(state, t)[2]
        o[:, :, t] = torch.einsum("bhkv,bhk->bhv", state, q[:, :, t])
    if s["op"] == "gated_fwd":
        o = _gather(s, o) if s["ends"] else o
        return (o, state) if s["S0"] is not None else (o,)
    do = _rows(s, ("dO",), torch.float64)[0]
    grad = torch.zeros_like(state) if s["dS"] is None else s["dS"].double()
    dq, dk, dvv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for t0 in sorted(marks, reverse=True):
        state, kept = marks[t0], []
        for t in range(t0, min(t0 + seg, length)):
            kept.append(token(state, t))
            state = kept[-1][2]
        for t in range(t0 + len(kept) - 1, t0 - 1, -1):
            faded, r, new = kept[t - t0]
            kt, al, dot = k[:, :, t], alpha[:, :, t, None], do[:, :, t]
            grad = grad + q[:, :, t][..., None] * dot[..., None, :]
            dq[:, :, t] = torch.einsum("bhkv,bhv->bhk", new, dot)
            gk, gr = torch.einsum("bhkv,bhk->bhv", grad, kt), torch.einsum("bhkv,bhv->bhk", grad, r)
            da = (kt * gr).sum(-1)
            dr = al * gk
            dvv[:, :, t] = dr
            dk[:, :, t] = al * gr - torch.einsum("bhkv,bhv->bhk", faded, dr)
            if s["mode"] == "exact":
                x = beta[:, :, t] * lam[:, :, t]
                few = beta[:, :, t] ** 2 * (-0.5 + x / 3 - x ** 2 / 8 + x ** 3 / 30 - x ** 4 / 144)
                dl = torch.where(x > 1e-2, (x * (-x).exp() + torch.expm1(-x)) / lam[:, :, t].clamp_min(1e-300) ** 2, few)
                dk[:, :, t] += 2 * (da * dl)[..., None] * kt
                db[:, :, t] = da * (-x).exp()
            else:
                db[:, :, t] = da
            grad = grad - kt[..., None] * dr[..., None, :]
            dg[:, :, t] = (grad * faded).sum((-1, -2))
            grad = grad * f[:, :, t, None, None]
    if rep > 1:
        dq, dk = (x.unflatten(1, (-1, rep)).sum(2) for x in (dq, dk))
    out = (dq, dk, dvv, dg, db)
    out = tuple(_gather(s, x) for x in out) if s["ends"] else out
    return out + ((grad,) if s["S0"] is not None else ())
