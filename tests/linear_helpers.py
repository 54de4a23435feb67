"""Float64 forms of moe_linear and its gradient, and bounds on the device's
error that count its roundings:
  * fp32 accumulation of K products: (K + 8) 2^-24 sum|a b|;
  * activations: |act'| <= 1.13, and their own evaluation (exp, erf, divide)
    within REL of the value; slopes within REL (1 + |z|);
  * dz and stored outputs rounded to the type: eps / 2 relative."""

import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}    # eps / 2
REL = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -17}
LIP = 1.13


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + \
            z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def clamped(z, u, limit):
    if limit > 0:
        return z.clamp(max=limit), u.clamp(-limit, limit), z <= limit, u.abs() <= limit
    yes = torch.ones_like(z, dtype=torch.bool)
    return z, u, yes, yes


def product(a, b):
    """a @ b.T in float64 and its fp32 accumulation bound."""
    a, b = a.double(), b.double()
    return a.mm(b.t().contiguous()), (a.shape[1] + 8) * 2.0 ** -24 * a.abs().mm(b.abs().t().contiguous())


def forward(c, x, w, bias=None, residual=None, w_up=None, bias_up=None):
    """(y, bound, z, dz, u, du): outputs, pre-activations and their bounds."""
    dt = x.dtype
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -24 * z.abs()
    u = eu = None
    if c.activation == "swiglu":
        u, eu = product(x, w_up)
        if bias_up is not None:
            u = u + bias_up.double()
            eu = eu + 2.0 ** -24 * u.abs()
        g, v, _, _ = clamped(z, u, c.limit)
        y = g / (1 + torch.exp(-g)) * v
        tol = LIP * v.abs() * ez + g.abs() * eu + REL[dt] * y.abs()
    else:
        y = act(z, c.activation)
        tol = LIP * ez + REL[dt] * y.abs()
    if residual is not None:
        y = y + residual.double()
        tol = tol + 2.0 ** -23 * y.abs()
    return y, tol + HALF[dt] * y.abs() + 1e-30, z, ez, u, eu


def backward(c, dy, x, w, z=None, w_up=None, u=None):
    """{name: (gradient, bound)} from the saved pre-activations as given."""
    dt = x.dtype
    half, rel = HALF[dt], REL[dt]
    d = dy.double()
    if c.activation == "swiglu":
        z, u = z.double(), u.double()
        g, v, on, on_up = clamped(z, u, c.limit)
        s = 1 / (1 + torch.exp(-g))
        dz = torch.where(on, d * v * s * (1 + g * (1 - s)), torch.zeros_like(d))
        du = torch.where(on_up, d * g * s, torch.zeros_like(d))
        ez = (d * v).abs() * rel * (1 + g.abs()) * on
        eu = du.abs() * rel
        parts = [("", dz, ez, w), ("_up", du, eu, w_up)]
    else:
        if c.activation == "none":
            dz, ez = d, torch.zeros_like(d)
        else:
            z = z.double()
            sl = slope(z, c.activation)
            dz = d * sl
            ez = d.abs() * rel * (1 + z.abs()) * (sl != 0)
        parts = [("", dz, ez, w)]
    out = {}
    dx = ex = 0.0
    for tag, g, e, wt in parts:
        r = e if c.activation == "none" else e + half * g.abs()   # dz as the products see it
        p, q = product(g, wt.t())
        dx, ex = dx + p, ex + q + r.mm(wt.double().abs())
        p, q = product(g.t(), x.t())
        out["dw" + tag] = (p, q + r.t().mm(x.double().abs()) + half * p.abs() + 1e-30)
        b = g.sum(0)
        out["dbias" + tag] = (b, e.sum(0) + (g.shape[0] + 8) * 2.0 ** -24 * g.abs().sum(0) +
                              half * b.abs() + 1e-30)
    out["dx"] = (dx, ex + half * dx.abs() + 1e-30)
    return out


def check(name, got, want, tol):
    assert torch.isfinite(got.double()).all(), name
    err = (got.double() - want).abs()
    if err.numel() == 0:
        return
    bad = (err > tol).sum().item()
    worst = (err / tol).max().item()
    print(f"[linear] {name}: worst {worst:.3f} of its bound", flush=True)
    assert bad == 0, f"{name}: {bad} of {err.numel()} past their bound, worst {worst:.2f} x"
