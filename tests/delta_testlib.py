"""Plain float64 forms of the gated delta rule and of the norm, on the CPU.

Written with torch operations token by token, so that autograd gives the
gradients of the definition itself.
"""
from __future__ import annotations

import torch


def delta_inputs(batch, seqlen, heads, groups, headdim, dstate, io, seed, decay="mixed", state=True):
    """CPU inputs: unit rows of q and k as a layer's norm gives them, values in
    the I/O type; decay "mixed" (0.02 to 3 per token), "slow" or "none"."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    x = {"q": unit(n(batch, seqlen, groups, dstate)).to(dt), "k": unit(n(batch, seqlen, groups, dstate)).to(dt),
         "v": n(batch, seqlen, heads, headdim).to(dt),
         "beta": torch.sigmoid(n(batch, seqlen, heads)).float(),
         "h0": (0.5 * n(batch, heads, headdim, dstate)).float() if state else None,
         "dout": n(batch, seqlen, heads, headdim).to(dt),
         "dend": (0.5 * n(batch, heads, headdim, dstate)).float() if state else None}
    g = {"mixed": -torch.exp(n(batch, seqlen, heads) - 1.5), "slow": -1e-3 * n(batch, seqlen, heads).abs(),
         "none": torch.zeros(batch, seqlen, heads, dtype=torch.float64)}[decay]
    x["g"] = g.float()
    return x


def delta_ref(q, k, v, g, beta, scale, h0=None):
    """(out, end state) in float64."""
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    batch, seqlen, heads, headdim = v.shape
    rep = heads // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    s = (torch.zeros(batch, heads, headdim, q.shape[3], dtype=torch.float64) if h0 is None else h0.double())
    out = []
    for t in range(seqlen):
        s = s * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhpn,bhn->bhp", s, k[:, t]))
        s = s + u[..., None] * k[:, t, :, None, :]
        out.append(scale * torch.einsum("bhpn,bhn->bhp", s, q[:, t]))
    return (torch.stack(out, 1) if out else v.clone()), s


def delta_grads(x, scale):
    """Gradients of sum(dout out) + sum(dend end state) by autograd in float64."""
    names = ("q", "k", "v", "g", "beta") + (("h0",) if x["h0"] is not None else ())
    leaf = {n: x[n].double().requires_grad_() for n in names}
    out, end = delta_ref(leaf["q"], leaf["k"], leaf["v"], leaf["g"], leaf["beta"], scale, leaf.get("h0"))
    loss = (out * x["dout"].double()).sum()
    if x["dend"] is not None:
        loss = loss + (end * x["dend"].double()).sum()
    got = torch.autograd.grad(loss, [leaf[n] for n in names])
    return dict(zip(names, got))


def norm_ref(x, weight, bias, z, eps, mode):
    """(out, mean, rstd) in float64."""
    x = x.double()
    mean = x.mean(-1) if mode == "layer" else None
    xc = x - mean[..., None] if mean is not None else x
    rstd = ((xc * xc).mean(-1) + eps) ** -0.5
    y = xc * rstd[..., None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    if z is not None:
        y = y * z.double() * torch.sigmoid(z.double())
    return y, mean, rstd
