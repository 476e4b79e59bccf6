"""Cases of the gated delta rule (forward, backward, one-token step) and of the normalisation (forward, backward).

The plain forms below are elementary torch operations in float32 (float64 for the sums of the log decays and the
triangular inverse); ``exact`` walks the definitions token by token in float64.  With ``own`` set, ``run`` makes the
calls of the library's binding.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64
_IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def _delta(op, name, io, batch, seqlen, heads, groups, headdim, dstate, **more):
    c = dict(name=name, op=op, io=io, batch=batch, seqlen=seqlen, heads=heads, groups=groups, headdim=headdim,
             dstate=dstate)
    c.update(more)
    return c


def _norm(op, name, io, rows, dim, mode, gate, bias):
    return dict(name=name, op=op, io=io, rows=rows, dim=dim, mode=mode, gate=gate, bias=bias)


def listed():
    return [
        # a short prompt appended to a running sequence: latency counts
        _delta("delta_fwd", "delta_fwd_short", "bf16", 1, 37, 8, 4, 64, 64, state=True),
        # one layer of a model with 4096 inner channels, two value heads to a key head
        _delta("delta_fwd", "delta_fwd_layer", "bf16", 8, 2048, 32, 16, 128, 128, state=True),
        # one long document, few heads
        _delta("delta_fwd", "delta_fwd_long", "bf16", 1, 32768, 16, 16, 64, 128, state=True),
        # float32 with sizes that no tile divides
        _delta("delta_fwd", "delta_fwd_f32_odd", "f32", 3, 301, 6, 3, 40, 48, state=True),
        # the training step of the same layer
        _delta("delta_bwd", "delta_bwd_layer", "bf16", 4, 2048, 32, 16, 128, 128, state=False),
        # a truncated-backpropagation segment: a start state, a gradient of the end state, a ragged tail
        _delta("delta_bwd", "delta_bwd_segment", "bf16", 2, 333, 4, 4, 64, 64, state=True),
        # decoding with a full batch
        _delta("delta_step", "delta_step_b256", "bf16", 256, 1, 32, 16, 128, 128, state=True),
        # decoding one sequence
        _delta("delta_step", "delta_step_b1", "bf16", 1, 1, 16, 16, 64, 128, state=True),
        # the gated norm of each head's output, after the layer above
        _norm("norm_fwd", "norm_fwd_heads", "bf16", 8 * 2048 * 32, 128, "rms", True, False),
        # a block's layer norm while decoding
        _norm("norm_fwd", "norm_fwd_decode", "bf16", 256, 2048, "layer", False, True),
        # a block's layer norm in training
        _norm("norm_bwd", "norm_bwd_block", "bf16", 8 * 2048, 2048, "layer", False, True),
        # float32, odd row length, with the gate
        _norm("norm_bwd", "norm_bwd_f32_odd", "f32", 2049, 515, "layer", True, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_bwd", "delta_step", "norm_fwd", "norm_bwd"])
    io = "f32" if rng.random() < 0.25 else "bf16"
    if op.startswith("norm"):
        dim = rng.choice([64, 128, 768, 1024, 2048, 4096]) if rng.random() < 0.6 else _log_int(rng, 8, 5000)
        rows = min(_log_int(rng, 1, 100000), 60_000_000 // dim)
        return dict(op=op, io=io, rows=rows, dim=dim, mode=rng.choice(["layer", "rms"]), gate=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
    groups = rng.choice([1, 2, 3, 4, 8, 16])
    heads = groups * rng.choice([1, 2, 3])
    if io == "bf16" and rng.random() < 0.7:
        headdim, dstate = rng.choice([64, 128]), rng.choice([64, 128])
    else:
        headdim, dstate = rng.randint(8, 128), rng.randint(8, 128)
    if op == "delta_step":
        batch, seqlen = _log_int(rng, 1, 256), 1
    else:
        batch, seqlen = rng.randint(1, 8), _log_int(rng, 1, 4096)
        if io == "f32":
            batch, seqlen = min(batch, 3), min(seqlen, 700)
    return dict(op=op, io=io, batch=batch, seqlen=seqlen, heads=heads, groups=groups, headdim=headdim, dstate=dstate,
                state=rng.random() < 0.7 or op == "delta_step")


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    io = _IO[case["io"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    s = {"case": case, "op": case["op"]}
    if case["op"].startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        s["x"] = (normal(rows, dim) * 1.5 + 0.3).to(io)
        s["weight"] = 1 + 0.2 * normal(dim)
        s["bias"] = 0.1 * normal(dim) if case["bias"] else None
        s["z"] = normal(rows, dim).to(io) if case["gate"] else None
        s["eps"] = 1e-5
        s["mode"] = case["mode"]
        if case["op"] == "norm_bwd":
            s["dout"] = normal(rows, dim).to(io)
            # the forward pass's statistics, as it leaves them
            x = s["x"].double()
            mean = x.mean(1) if case["mode"] == "layer" else torch.zeros(rows, dtype=torch.float64, device=DEV)
            s["mean"] = mean.float() if case["mode"] == "layer" else None
            s["rstd"] = (((x - mean[:, None]) ** 2).mean(1) + s["eps"]).rsqrt().float()
        return s
    b, l, h, gr = case["batch"], case["seqlen"], case["heads"], case["groups"]
    p, n = case["headdim"], case["dstate"]
    q, k = normal(b, l, gr, n), normal(b, l, gr, n)
    s["q"] = (q / (q * q).sum(-1, keepdim=True).sqrt()).to(io)  # unit rows, as the layer's norm gives them
    s["k"] = (k / (k * k).sum(-1, keepdim=True).sqrt()).to(io)
    s["v"] = normal(b, l, h, p).to(io)
    # log decay -A Delta with A in [1, 16] and Delta = softplus(raw + inverse softplus of [1e-3, 1e-1])
    dt0 = torch.exp(uniform(h) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    raw = 0.5 * normal(b, l, h) + dt0 + torch.log(-torch.expm1(-dt0))
    s["g"] = -(1 + 15 * uniform(h)) * (raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs())))
    s["beta"] = torch.sigmoid(normal(b, l, h))
    s["scale"] = n ** -0.5
    state = 0.3 * normal(b, h, p, n) if case["state"] else None
    if case["op"] == "delta_step":
        for name in ("q", "k", "v", "g", "beta"):
            s[name] = s[name][:, 0].contiguous()
        s["state"] = state
    elif case["op"] == "delta_fwd":
        s["state"] = state
    else:
        s["h0"] = state
        s["dstate_end"] = 0.3 * normal(b, h, p, n) if case["state"] else None
        s["dout"] = normal(b, l, h, p).to(io)
    return s


# ------------------------------------------------------------- plain forms
def _heads_of(x, heads):
    """(batch, chunks, C, groups, n) -> float32 (batch, chunks, heads, C, n), groups repeated over their heads."""
    return x.float().transpose(2, 3).repeat_interleave(heads // x.shape[3], dim=2)


def _chunks(x, c):
    """(batch, seqlen, ...) -> (batch, chunks, c, ...), zeros behind the end."""
    pad = -x.shape[1] % c
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    return x.reshape(x.shape[0], -1, c, *x.shape[2:])


def _prologue(s, c):
    """What every chunk needs and no state enters: float32, (batch, chunks, heads, ...)."""
    h = s["v"].shape[2]
    q, k = _heads_of(_chunks(s["q"], c), h), _heads_of(_chunks(s["k"], c), h)
    v = _chunks(s["v"], c).float().transpose(2, 3)
    beta = _chunks(s["beta"], c).transpose(2, 3)
    cum = _chunks(s["g"], c).transpose(2, 3).double().cumsum(-1)
    low = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    gam = torch.where(low, (cum[..., :, None] - cum[..., None, :]).masked_fill(~low, 0).exp().float(), 0)
    a = (gam * (k @ k.transpose(-1, -2))).tril(-1)
    # (I + a diag(beta))^-1 as the product of I + x^(2^i), x = -a diag(beta) nilpotent
    x = -(a * beta[..., None, :]).double()
    eye = torch.eye(c, dtype=torch.float64, device=q.device)
    inv = eye + x
    x = x @ x
    inv = inv @ (eye + x)
    x = x @ x
    inv = inv @ (eye + x)
    x = x @ x
    inv = inv @ (eye + x)
    x = x @ x
    inv = inv @ (eye + x)
    x = x @ x
    inv = (inv @ (eye + x)).float()
    qk = s["scale"] * gam * (q @ k.transpose(-1, -2))
    start = cum.exp().float()[..., None]                       # decay from the chunk's start to t
    end = (cum[..., -1:] - cum).exp().float()[..., None]       # decay from t to the chunk's end
    return q, k, v, beta[..., None], gam, a, inv, qk, start, end, start[..., -1:, :]


def _plain_delta_fwd(s, keep=False):
    v = s["v"]
    b, l, h, p = v.shape
    n = s["q"].shape[-1]
    q, k, v, beta, gam, a, inv, qk, start, end, whole = _prologue(s, CHUNK)
    state = s.get("h0") if keep else s["state"]
    st = torch.zeros(b, h, p, n, device=v.device) if state is None else state
    qs, ks, kw = s["scale"] * start * q, start * k, end * k
    out, states, rs = torch.empty_like(v), [], []
    for i in range(v.shape[1]):
        r = inv[:, i] @ (v[:, i] - ks[:, i] @ st.transpose(-1, -2))
        u = beta[:, i] * r
        out[:, i] = qs[:, i] @ st.transpose(-1, -2) + qk[:, i] @ u
        if keep:
            states.append(st)
            rs.append(r)
        st = whole[:, i] * st + u.transpose(-1, -2) @ kw[:, i]
    if keep:
        return states + [st], rs
    out = out.transpose(2, 3).reshape(b, -1, h, p)[:, :l].to(s["v"].dtype)
    if state is not None:
        state.copy_(st)
    return {"out": out, "state": state}


def _plain_delta_bwd(s):
    b, l, h, p = s["v"].shape
    gr, n = s["q"].shape[2:]
    io = s["v"].dtype
    states, rs = _plain_delta_fwd(s, keep=True)
    q, k, v, beta, gam, a, inv, qk, start, end, whole = _prologue(s, CHUNK)
    do = _chunks(s["dout"], CHUNK).float().transpose(2, 3)
    ds = torch.zeros_like(states[0]) if s["dstate_end"] is None else s["dstate_end"]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta, dg = torch.empty_like(beta), torch.empty_like(beta)
    for i in reversed(range(v.shape[1])):
        r, s0 = rs[i], states[i]
        u = beta[:, i] * r
        du = qk[:, i].transpose(-1, -2) @ do[:, i] + end[:, i] * (k[:, i] @ ds.transpose(-1, -2))
        dv[:, i] = inv[:, i].transpose(-1, -2) @ (beta[:, i] * du)
        e = du - a[:, i].transpose(-1, -2) @ dv[:, i]
        x = s["scale"] * gam[:, i] * (do[:, i] @ u.transpose(-1, -2))
        y = -(gam[:, i] * (dv[:, i] @ u.transpose(-1, -2))).tril(-1)
        dq[:, i] = s["scale"] * start[:, i] * (do[:, i] @ s0) + x @ k[:, i]
        left = y @ k[:, i] - start[:, i] * (dv[:, i] @ s0)
        right = x.transpose(-1, -2) @ q[:, i] + y.transpose(-1, -2) @ k[:, i] + end[:, i] * (u @ ds)
        dk[:, i] = left + right
        dbeta[:, i] = (e * r).sum(-1, keepdim=True)
        dcum = (q[:, i] * dq[:, i] + k[:, i] * (left - right)).double().sum(-1, keepdim=True)
        dcum[..., -1:, :] += (states[i + 1] * ds).double().sum((-1, -2))[..., None, None]
        dg[:, i] = dcum.flip(-2).cumsum(-2).flip(-2).float()
        ds = (whole[:, i] * ds + (s["scale"] * start[:, i] * do[:, i]).transpose(-1, -2) @ q[:, i]
              - (start[:, i] * dv[:, i]).transpose(-1, -2) @ k[:, i])

    def back(x, width):
        return x.transpose(2, 3).reshape(b, -1, h, width)[:, :l]

    def grouped(x):
        return back(x, n).reshape(b, l, gr, h // gr, n).sum(3).to(io)

    return {"dq": grouped(dq), "dk": grouped(dk), "dv": back(dv, p).to(io), "dg": back(dg, 1)[..., 0].contiguous(),
            "dbeta": back(dbeta, 1)[..., 0].contiguous(), "dh0": ds if s["h0"] is not None else None}


def _plain_delta_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[x].float().repeat_interleave(rep, 1) for x in ("q", "k"))
    st = s["state"] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (st * k[:, :, None, :]).sum(-1))
    st = st + u[..., None] * k[:, :, None, :]
    out = s["scale"] * (st * q[:, :, None, :]).sum(-1)
    s["state"].copy_(st)
    return {"out": out.to(s["v"].dtype), "state": s["state"]}


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1) if s["mode"] == "layer" else None
    xc = x - mean[:, None] if mean is not None else x
    rstd = ((xc * xc).mean(1) + s["eps"]).rsqrt()
    y = xc * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"out": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dout"].float()
    xh = (x - s["mean"][:, None] if s["mean"] is not None else x) * s["rstd"][:, None]
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        y = xh * s["weight"] + (s["bias"] if s["bias"] is not None else 0)
        sig = torch.sigmoid(z)
        dz = (dy * y * sig * (1 + z * (1 - sig))).to(s["x"].dtype)
        dy = dy * z * sig
    dh = dy * s["weight"]
    dx = dh - xh * (dh * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - dh.mean(1, keepdim=True)
    return {"dx": (dx * s["rstd"][:, None]).to(s["x"].dtype), "dz": dz, "dweight": (dy * xh).sum(0),
            "dbias": dy.sum(0) if s["bias"] is not None else None}


def _own(s):
    from selective_state_space_36_b200 import binding as lib

    op = s["op"]
    if op == "delta_fwd":
        out = lib.delta_rule_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], last_state=s["state"])
        return {"out": out, "state": s["state"]}
    if op == "delta_bwd":
        return lib.delta_rule_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], scale=s["scale"], h0=s["h0"],
                                  dlast_state=s["dstate_end"])
    if op == "delta_step":
        out = lib.delta_rule_update(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"])
        return {"out": out, "state": s["state"]}
    if op == "norm_fwd":
        out, mean, rstd = lib.norm_fwd(s["x"], s["weight"], s["bias"], z=s["z"], eps=s["eps"], mode=s["mode"])
        return {"out": out, "mean": mean, "rstd": rstd}
    return lib.norm_bwd(s["x"], s["weight"], s["dout"], s["rstd"], mean=s["mean"], bias=s["bias"], z=s["z"])


_PLAIN = {"delta_fwd": _plain_delta_fwd, "delta_bwd": _plain_delta_bwd, "delta_step": _plain_delta_step,
          "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"].startswith("norm"):
        m, d = case["rows"] * case["dim"], case["dim"]
        if case["op"] == "norm_fwd":
            byt = m * e * (3 if case["gate"] else 2) + 4 * case["rows"] * (2 if case["mode"] == "layer" else 1)
            return {"bytes": byt + 4 * d * (2 if case["bias"] else 1), "flops": m * (12 if case["gate"] else 8)}
        byt = m * e * (5 if case["gate"] else 3) + 4 * case["rows"] * (2 if case["mode"] == "layer" else 1)
        return {"bytes": byt + 4 * d * (4 if case["bias"] else 2), "flops": m * (24 if case["gate"] else 14)}
    t = case["batch"] * case["seqlen"]
    h, gr, p, n = case["heads"], case["groups"], case["headdim"], case["dstate"]
    held = 4 * case["batch"] * h * p * n
    if case["op"] == "delta_bwd":
        byt = t * (e * (4 * gr * n + 3 * h * p) + 16 * h) + (3 * held if case["state"] else 0)
        return {"bytes": byt, "flops": t * h * 22 * p * n}
    byt = t * (e * (2 * gr * n + 2 * h * p) + 8 * h) + (2 * held if case["state"] else 0)
    return {"bytes": byt, "flops": t * h * 8 * p * n}


# ------------------------------------------------------------------- exact
def _walk(st, s, lo, hi, keep):
    """Tokens lo..hi of the definition in float64, from the state st: (state, outputs, states before each, r)."""
    outs, before, rs = [], [], []
    for t in range(lo, hi):
        if keep:
            before.append(st)
        st = st * s["a"][:, t, :, None, None]
        r = s["v"][:, t] - torch.einsum("bhpn,bhn->bhp", st, s["k"][:, t])
        st = st + (s["beta"][:, t, :, None] * r)[..., None] * s["k"][:, t, :, None, :]
        rs.append(r)
        outs.append(s["scale"] * torch.einsum("bhpn,bhn->bhp", st, s["q"][:, t]))
    return st, outs, before, rs


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    if case["op"] == "delta_step":
        for name in ("q", "k", "v", "g", "beta"):
            s[name] = s[name][:, None]
    rep = case["heads"] // case["groups"]
    d = {"scale": s["scale"], "v": s["v"].double(), "beta": s["beta"].double(), "a": s["g"].double().exp(),
         "q": s["q"].double().repeat_interleave(rep, 2), "k": s["k"].double().repeat_interleave(rep, 2)}
    b, l, h, p = s["v"].shape
    zero = torch.zeros(b, h, p, case["dstate"], dtype=torch.float64, device=DEV)
    if case["op"] != "delta_bwd":
        st, outs, _, _ = _walk(zero if s["state"] is None else s["state"].double(), d, 0, l, False)
        out = torch.stack(outs, 1) if case["op"] == "delta_fwd" else outs[0]
        return {"out": out, "state": st if s["state"] is not None else None}
    # backward: states at every 32nd token, the others walked again from there
    step = 32
    st, marks = zero if s["h0"] is None else s["h0"].double(), []
    for lo in range(0, l, step):
        marks.append(st)
        st = _walk(st, d, lo, min(l, lo + step), False)[0]
    ds = zero if s["dstate_end"] is None else s["dstate_end"].double()
    do = s["dout"].double()
    got = {x: [None] * l for x in ("dq", "dk", "dv", "dg", "dbeta")}
    for lo in reversed(range(0, l, step)):
        end, _, before, rs = _walk(marks[lo // step], d, lo, min(l, lo + step), True)
        after = before[1:] + [end]
        for t in reversed(range(lo, min(l, lo + step))):
            old, new, r = before[t - lo], after[t - lo], rs[t - lo]
            k, a, beta = d["k"][:, t], d["a"][:, t, :, None], d["beta"][:, t, :, None]
            got["dq"][t] = s["scale"] * torch.einsum("bhpn,bhp->bhn", new, do[:, t])
            ds = ds + (s["scale"] * do[:, t])[..., None] * d["q"][:, t, :, None, :]
            du = torch.einsum("bhpn,bhn->bhp", ds, k)
            got["dbeta"][t] = (du * r).sum(-1)
            got["dv"][t] = dr = beta * du
            got["dk"][t] = (torch.einsum("bhpn,bhp->bhn", ds, beta * r)
                            - a * torch.einsum("bhpn,bhp->bhn", old, dr))
            ds = a[..., None] * (ds - dr[..., None] * k[:, :, None, :])
            got["dg"][t] = (ds * old).sum((-1, -2))
    got = {x: torch.stack(y, 1) for x, y in got.items()}
    for x in ("dq", "dk"):
        got[x] = got[x].reshape(b, l, case["groups"], rep, -1).sum(3)
    got["dh0"] = ds if s["h0"] is not None else None
    return got


def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    mean = x.mean(1) if case["mode"] == "layer" else None
    xc = x - mean[:, None] if mean is not None else x
    rstd = 1 / torch.sqrt((xc ** 2).mean(1) + s["eps"])
    if case["op"] == "norm_bwd":  # the statistics are inputs there
        rstd = s["rstd"].double()
        xc = x - s["mean"].double()[:, None] if mean is not None else x
    bias = s["bias"].double() if s["bias"] is not None else None
    xh = xc * rstd[:, None]
    y = xh * w + bias if bias is not None else xh * w
    z = s["z"].double() if s["z"] is not None else None
    gate = z / (1 + torch.exp(-z)) if z is not None else None
    if case["op"] == "norm_fwd":
        return {"out": y * gate if z is not None else y, "mean": mean, "rstd": rstd}
    do, dz = s["dout"].double(), None
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        dz = do * y * (sig + z * sig * (1 - sig))
        do = do * gate
    dxh = do * w
    dx = dxh - xh * (dxh * xh).sum(1, keepdim=True) / case["dim"]
    if mean is not None:
        dx = dx - dxh.sum(1, keepdim=True) / case["dim"]
    return {"dx": dx * rstd[:, None], "dz": dz, "dweight": (do * xh).sum(0),
            "dbias": do.sum(0) if bias is not None else None}
