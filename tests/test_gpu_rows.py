"""Token rows to experts and back on the GPU: dispatch, combine and their gradients
against float64 forms."""

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C
from tests import train_helpers as H

pytestmark = pytest.mark.gpu

# tokens, width, slots, experts, share of dropped pairs
CASES = [(1, 8, 1, 1, 0.0), (1, 7168, 8, 256, 0.0), (3, 7, 2, 4, 0.0), (5, 1, 3, 4, 0.2),
         (17, 9, 16, 16, 0.1), (64, 64, 2, 8, 0.0), (203, 1001, 3, 16, 0.3), (257, 2048, 4, 64, 0.02),
         (1000, 192, 5, 7, 0.5), (31, 4, 6, 12, 1.0), (40, 3, 7, 9, 0.1), (129, 520, 9, 24, 0.1)]


def config(d, k, E, dtype):
    return C.MoEConfig(dim=d, n_routed_experts=E, n_activated_experts=k, moe_inter_dim=64,
                       act_dtype=dtype, expert_dtype=dtype)


def inputs(T, d, k, E, dropped, dtype, spare=3):
    g, dt = H.gen(T * 31 + d * 7 + k), H.TDT[dtype]
    inverse, R = H.permutation(T, k, E, g, dropped)
    return (inverse, R, H.normal(g, dt, T, d), H.normal(g, dt, R + spare, d),
            torch.rand((T, k), generator=g) + 0.01, H.normal(g, dt, T, d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,k,E,dropped", CASES)
def test_rows(gpu, T, d, k, E, dropped, dtype):
    print(f"[rows] T={T} d={d} k={k} E={E} dropped={dropped} {dtype}", flush=True)
    cfg, dt = config(d, k, E, dtype), H.TDT[dtype]
    half = H.HALF[dt]
    inverse, R, x, rows, w, add = inputs(T, d, k, E, dropped, dtype)
    there = inverse >= 0
    dev = [t.to(gpu) for t in (inverse, x, rows, w, add)]
    inv_d, x_d, rows_d, w_d, add_d = dev
    # dispatch: copies; rows of no pair are left as they were
    out = torch.full((R + 3, d), -7.0, dtype=dt, device=gpu)
    B.moe_dispatch(cfg, x_d, inv_d, T, out)
    want = torch.full((R + 3, d), -7.0, dtype=dt)
    want[inverse[there].long()] = x.unsqueeze(1).expand(T, k, d)[there]
    assert torch.equal(out.cpu(), want)
    # its gradient, and combine with and without what is added
    got, _ = H.gathered(rows, inverse)
    y = torch.empty((T, d), dtype=dt, device=gpu)
    tol = lambda terms, v: (k + 2) * 2.0 ** -24 * terms + half * v.abs() + 1e-30
    B.moe_dispatch_backward(cfg, rows_d, inv_d, T, y)
    v = got.sum(1)
    H.check("dx", y, v, tol(got.abs().sum(1), v))
    wd = (w.double() * there).unsqueeze(2)
    for a, a_d in ((None, None), (add, add_d)):
        B.moe_combine(cfg, rows_d, inv_d, w_d, T, y, add=a_d)
        v, terms = (wd * got).sum(1), (wd * got).abs().sum(1)
        if a is not None:
            v, terms = v + a.double(), terms + a.double().abs()
        H.check("y", y, v, tol(terms, v))
    # the gradient of combine, both and each alone
    drows = torch.full((R + 3, d), -7.0, dtype=dt, device=gpu)
    dw = torch.full((T, k), -7.0, device=gpu)
    B.moe_combine_backward(cfg, x_d, rows_d, inv_d, w_d, T, drows=drows, dweights=dw)
    want = torch.full((R + 3, d), -7.0, dtype=torch.float64)
    want[inverse[there].long()] = (w.double().unsqueeze(2) * x.double().unsqueeze(1))[there]
    H.check("drows", drows, want, (2.0 ** -24 + half) * want.abs() + 1e-30)
    assert torch.equal(drows[R:].cpu(), torch.full((3, d), -7.0, dtype=dt))
    dots = got * x.double().unsqueeze(1)
    H.check("dweights", dw, dots.sum(2), (d + 8) * 2.0 ** -24 * dots.abs().sum(2) + 1e-30)
    assert (dw.cpu()[~there] == 0).all()
    alone = torch.full_like(drows, -7.0)
    B.moe_combine_backward(cfg, x_d, None, inv_d, w_d, T, drows=alone)
    assert torch.equal(alone, drows)
    alone = torch.empty_like(dw)
    B.moe_combine_backward(cfg, x_d, rows_d, inv_d, None, T, dweights=alone)
    assert torch.equal(alone, dw)
    for t, h in zip(dev, (inverse, x, rows, w, add)):        # inputs untouched
        assert torch.equal(t.cpu(), h)


# 1024 tokens and rows of 192 pieces of 16 bytes (1529 columns in bf16, 765 in fp32) take
# a workgroup a token: both sides of either border, odd widths, every number of slots
MANY = [(1024, 1529, 1, 4, 0.0), (1024, 1528, 2, 4, 0.1), (1023, 1601, 3, 8, 0.1),
        (1024, 1601, 3, 8, 0.1), (1027, 765, 4, 8, 0.0), (1024, 764, 4, 8, 0.1),
        (1025, 801, 5, 8, 0.3), (1024, 4099, 2, 8, 0.0), (1031, 1601, 8, 16, 0.5),
        (1024, 1537, 7, 9, 0.02), (1100, 2048, 9, 16, 0.1), (1040, 1544, 16, 24, 0.3),
        (2000, 1600, 6, 12, 1.0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,k,E,dropped", MANY)
def test_rows_of_many_tokens(gpu, T, d, k, E, dropped, dtype):
    test_rows(gpu, T, d, k, E, dropped, dtype)


def test_rows_out_of_range_take_no_part(gpu):
    cfg = config(24, 3, 8, "bf16")
    inverse, R, x, rows, w, _ = inputs(50, 24, 3, 8, 0.0, "bf16", spare=0)
    good = inverse.clone()
    for i, bad in enumerate((R, R + 5, -1, -2, 2 ** 31 - 1, -2 ** 31)):
        inverse[i * 7, i % 3] = bad
        good[i * 7, i % 3] = -1
    outs = []
    for inv in (inverse.to(gpu), good.to(gpu)):
        out = torch.zeros((R, 24), dtype=torch.bfloat16, device=gpu)
        y, dw, dr = torch.empty((50, 24), dtype=torch.bfloat16, device=gpu), torch.empty((50, 3), device=gpu), torch.zeros_like(out)
        B.moe_dispatch(cfg, x.to(gpu), inv, 50, out)
        B.moe_combine(cfg, rows.to(gpu), inv, w.to(gpu), 50, y)
        B.moe_combine_backward(cfg, x.to(gpu), rows.to(gpu), inv, w.to(gpu), 50, drows=dr, dweights=dw)
        outs.append([t.cpu() for t in (out, y, dw, dr)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_values_that_are_not_finite_stay_in_their_rows(gpu):
    cfg = config(16, 2, 4, "f32")
    inverse, R, x, rows, w, _ = inputs(20, 16, 2, 4, 0.3, "f32", spare=0)
    hole = (inverse == -1).any()
    assert hole
    row = int(inverse[4].max())
    assert row >= 0
    rows[row, 3], rows[row, 5] = float("nan"), float("inf")
    y = torch.empty((20, 16), device=gpu)
    B.moe_combine(cfg, rows.to(gpu), inverse.to(gpu), w.to(gpu), 20, y)
    bad = ~torch.isfinite(y.cpu())
    assert bad[4, 3] and bad[4, 5] and bad.sum() == 2


@pytest.mark.parametrize("call", ["dispatch", "combine"])
def test_no_sorted_rows(gpu, call):
    cfg = config(16, 2, 4, "bf16")
    none = torch.empty((0, 16), dtype=torch.bfloat16, device=gpu)
    inv = torch.full((5, 2), -1, dtype=torch.int32, device=gpu)
    y = torch.full((5, 16), 3.0, dtype=torch.bfloat16, device=gpu)
    if call == "dispatch":
        B.moe_dispatch(cfg, y, inv, 5, none)
        B.moe_dispatch_backward(cfg, none, inv, 5, y)
    else:
        B.moe_combine(cfg, none, inv, torch.ones((5, 2), device=gpu), 5, y)
    assert (y == 0).all()


def test_offsets_past_32_bits(gpu):
    """Sorted rows whose bytes and elements pass 32 bits."""
    d, R = 7168, 620_000                                     # 4.4e9 elements
    cfg = config(d, 2, 4, "bf16")
    rows = torch.empty((R, d), dtype=torch.bfloat16, device=gpu)
    inv = torch.tensor([[R - 1, 0], [R - 2, 300_000], [599_187, -1]], dtype=torch.int32)
    for r in inv[inv >= 0].tolist():
        rows[r] = float(r % 251 + 1)
    w = torch.tensor([[1.0, 2.0], [3.0, 4.0], [0.5, 9.0]])
    y = torch.empty((3, d), dtype=torch.bfloat16, device=gpu)
    B.moe_combine(cfg, rows, inv.to(gpu), w.to(gpu), 3, y)
    want = torch.where(inv >= 0, w * (inv % 251 + 1), 0.0).sum(1)
    assert torch.equal(y.cpu(), want.to(torch.bfloat16).unsqueeze(1).expand(3, d))
    x = torch.arange(3, device=gpu).to(torch.bfloat16).add(5).unsqueeze(1).expand(3, d).contiguous()
    B.moe_dispatch(cfg, x, inv.to(gpu), 3, rows)
    for t in range(3):
        for r in inv[t].tolist():
            if r >= 0:
                assert (rows[r] == 5 + t).all()
