"""Float64 forms of what trains the MoE layer, and bounds on the device's error that
count its roundings:
  * fp32 sums of n products: (n + 8) 2^-24 sum|a b|;
  * SwiGLU and its slopes: their own evaluation within REL of the value;
  * stored results, and h, dz and du as the products take them: eps / 2 relative."""

import math

import torch

from tests.linear_helpers import HALF, LIP, REL

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, dt, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dt)


# ---- rows ------------------------------------------------------------------

def permutation(T, k, E, g, dropped=0.0):
    """(inverse [T, k], rows): a stable sort by expert, some pairs dropped."""
    expert = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]) if T else \
        torch.zeros((0, k), dtype=torch.long)
    expert = torch.where(torch.rand((T, k), generator=g) < dropped, E, expert).reshape(-1)
    order = expert.sort(stable=True)[1]
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(T * k)
    inverse[expert == E] = -1
    return inverse.reshape(T, k).to(torch.int32), int((expert < E).sum())


def gathered(rows, inverse):
    """rows[inverse] [T, k, d] in float64, zeros where there is none; and where there is."""
    R = rows.shape[0]
    there = (inverse >= 0) & (inverse < R)
    out = torch.zeros((*inverse.shape, rows.shape[1]), dtype=torch.float64)
    out[there] = rows.double()[inverse[there].long()]
    return out, there


# ---- 8-bit checkpoints -----------------------------------------------------

def code_values():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        a = math.nan if (c & 127) == 127 else a
        v.append(-a if c & 128 else a)
    return torch.tensor(v, dtype=torch.float64)


VALUES = code_values()


def encode(src, limit=0.0):
    """(codes, scales) of a matrix by the definition, code by code."""
    v = src.double()
    rows, cols = v.shape
    blocks = -(-cols // 32)
    mags = VALUES[:127]
    codes = torch.empty((rows, cols), dtype=torch.uint8)
    scales = torch.empty((rows, blocks), dtype=torch.uint8)
    for b in range(blocks):
        w = v[:, 32 * b:32 * b + 32]
        fine = torch.isfinite(w)
        top = torch.where(fine, w.abs(), 0.0).amax(dim=1)
        x = torch.zeros(rows, dtype=torch.int64)
        for r in range(rows):
            if top[r] > 0:
                m, e = math.frexp(float(top[r]))
                x[r] = max(-127, e - 9 + (1 if m > 0.875 else 0))
        a = w.abs() * torch.exp2(-x.double()).unsqueeze(1)
        a = torch.where(fine, a, 0.0)
        hi = torch.searchsorted(mags, a.contiguous()).clamp(max=126)    # first code not below
        lo = (hi - 1).clamp(min=0)
        below, above = a - mags[lo], mags[hi] - a
        code = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
        if limit > 0:
            edge = limit * torch.exp2(-x.double()).unsqueeze(1)
            code = torch.where((a > edge) & (mags[code] <= edge), hi, code)
            code = torch.where((a <= edge) & (mags[code] > edge), lo, code)
        code = torch.where(fine, code, 127) + 128 * torch.signbit(w)
        codes[:, 32 * b:32 * b + 32] = code.to(torch.uint8)
        scales[:, b] = (x + 127).to(torch.uint8)
    return codes, scales


def encode_whole(src, limit=0.0):
    """encode() of finite values in whole blocks at once, where the matrix is."""
    rows, cols = src.shape
    v = torch.zeros((rows, -(-cols // 32) * 32), dtype=torch.float64, device=src.device)
    v[:, :cols] = src
    v = v.reshape(rows, -1, 32)
    m, e = torch.frexp(v.abs().amax(dim=2))
    x = torch.where(m > 0, (e - 9 + (m > 0.875)).clamp(min=-127), 0)
    unit = torch.exp2(x.double()).unsqueeze(2)
    mags, a = VALUES[:127].to(src.device), v.abs() / unit
    hi = torch.searchsorted(mags, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - mags[lo], mags[hi] - a
    code = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    if limit > 0:
        edge = limit / unit
        code = torch.where((a > edge) & (mags[code] <= edge), hi, code)
        code = torch.where((a <= edge) & (mags[code] > edge), lo, code)
    code = (code + 128 * torch.signbit(v)).to(torch.uint8).reshape(rows, -1)[:, :cols]
    return code.contiguous(), (x + 127).to(torch.uint8)


def decode(codes, scales):
    unit = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)[:, :codes.shape[1]]
    return VALUES[codes.long()] * unit


# ---- experts ---------------------------------------------------------------

def product(a, b):
    """a b^T in float64, and its fp32 accumulation's bound."""
    return a.mm(b.t()), (a.shape[1] + 8) * 2.0 ** -24 * a.abs().mm(b.abs().t())


def halves(z, u, limit):
    top = limit if limit > 0 else math.inf
    g, v = z.clamp(max=top), u.clamp(-top, top)
    return g, v, 1 / (1 + torch.exp(-g)), z <= top, u.abs() <= top


def experts_forward(x, wg, wu, wd, limit):
    """One expert: {name: (value, bound)} of z, u and y."""
    dt = x.dtype
    half, rel = HALF[dt], REL[dt]
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    z, ez = product(x, wg)
    u, eu = product(x, wu)
    g, v, q, _, _ = halves(z, u, limit)
    h = g * q * v
    eh = LIP * v.abs() * ez + g.abs() * eu + rel * h.abs()
    y, ey = product(h, wd)
    ey = ey + (eh + half * h.abs() + half * eh).mm(wd.abs().t())
    return {"z": (z, ez), "u": (u, eu), "y": (y, ey + half * (y.abs() + ey) + 1e-30)}


def experts_backward(x, wg, wu, wd, z, u, dy, limit):
    """One expert's gradients from the saved z and u (float64): {name: (value, bound)}."""
    dt = x.dtype
    half, rel = HALF[dt], REL[dt]
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    g, v, q, on, on_up = halves(z, u, limit)
    dh, eh = product(dy, wd.t())
    slope = v * q * (1 + g * (1 - q)) * on
    slope_up = g * q * on_up
    dz, du, h = dh * slope, dh * slope_up, g * q * v
    ez = slope.abs() * eh + (dh * v).abs() * rel * (1 + g.abs()) * on
    eu = slope_up.abs() * eh + du.abs() * rel
    rz, ru = ez + half * (dz.abs() + ez), eu + half * (du.abs() + eu)   # as the products take them
    rh = (rel + half) * h.abs()
    out = {}
    p, e = product(dz, wg.t())
    p2, e2 = product(du, wu.t())
    out["dx"] = p + p2, e + e2 + rz.mm(wg.abs()) + ru.mm(wu.abs())
    p, e = product(dz.t(), x.t())
    out["dw_gate"] = p, e + rz.t().mm(x.abs())
    p, e = product(du.t(), x.t())
    out["dw_up"] = p, e + ru.t().mm(x.abs())
    p, e = product(dy.t(), h.t())
    out["dw_down"] = p, e + dy.abs().t().mm(rh)
    return {n: (p, e + half * (p.abs() + e) + 1e-30) for n, (p, e) in out.items()}


def check(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, name
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    bad = int((err > tol).sum())
    worst = float((err / tol.clamp(min=1e-300)).max())
    print(f"[train] {name}: worst {worst:.3f} of its bound", flush=True)
    assert bad == 0, f"{name}: {bad} of {err.numel()} past their bound, worst {worst:.2f} x"
