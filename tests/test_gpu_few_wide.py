"""moe_forward_few on FP4 layers so wide that a row's scales go through LDS in
several pieces, at the width where its down launch changes form, and around the
size from which a gate has a launch of its own."""

from dataclasses import replace

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C
from tests import test_gpu_few as F

pytestmark = pytest.mark.gpu

W = C.SMALL_WORKLOADS


def wide(base, dim, inter):
    w = W[base]
    groups = dict(n_expert_groups=1, n_limited_groups=1)
    return replace(w, name=f"{base}_{dim}_{inter}", T=16, cfg=replace(
        w.cfg, dim=dim, moe_inter_dim=inter, n_routed_experts=8, n_activated_experts=2, **groups))


@pytest.mark.parametrize("base,dim,inter", [
    ("fp4_small", 8256, 64), ("fp4_small", 64, 8064), ("fp4_small", 128, 1792), ("fp4_small", 128, 1856),
    ("fp4_small", 7936, 64), ("fp4_small", 7968 // 64 * 64, 448),
    ("fp4_mx_small", 8320, 128), ("fp4_mx_small", 128, 8064), ("fp4_mx_small", 256, 1792),
    ("fp4_mx_small", 256, 1920)])
@pytest.mark.parametrize("T", [1, 9])
def test_wide_fp4(base, dim, inter, T, gpu, monkeypatch):
    wl = wide(base, dim, inter)
    monkeypatch.setitem(F.LAYERS, wl.name, wl)
    wl, cfg, run, plain = F.make(wl.name, T, gpu)
    print(f"[few] {wl.name} T={T}", flush=True)
    ws = torch.full((B.moe_few_workspace_size(cfg, T),), 0xFF, dtype=torch.uint8, device=gpu)
    y, _ = F.few(cfg, run, T, ws)
    torch.cuda.synchronize()
    F.check(wl, cfg, plain, T, y, ws, f"{wl.name} T={T}")
    tcfg, tlayer = B.pack_layer(cfg, run)
    yt, _ = F.few(tcfg, tlayer, T)
    torch.cuda.synchronize()
    assert torch.equal(y, yt)


@pytest.mark.parametrize("base,dim,experts", [
    ("tiny_fp32", 512, 64), ("tiny_fp32", 512, 65), ("tiny_fp32", 513, 64), ("tiny_fp32", 511, 33),
    ("v3_small", 1024, 64), ("v3_small", 1088, 64), ("v3_small", 1024, 72), ("v3_small", 64, 17)])
@pytest.mark.parametrize("T", [1, 16])
def test_gate_sizes(base, dim, experts, T, gpu, monkeypatch):
    """Around the largest gate whose logits need no launch of their own."""
    w = W[base]
    wl = replace(w, name=f"{base}_{dim}_{experts}", T=16, cfg=replace(
        w.cfg, dim=dim, n_routed_experts=experts, n_expert_groups=1, n_limited_groups=1,
        n_activated_experts=3))
    monkeypatch.setitem(F.LAYERS, wl.name, wl)
    wl, cfg, run, plain = F.make(wl.name, T, gpu)
    print(f"[few] {wl.name} T={T}", flush=True)
    ws = torch.full((B.moe_few_workspace_size(cfg, T),), 0xFF, dtype=torch.uint8, device=gpu)
    y, _ = F.few(cfg, run, T, ws)
    torch.cuda.synchronize()
    F.check(wl, cfg, plain, T, y, ws, f"{wl.name} T={T}")
