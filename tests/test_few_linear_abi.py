"""moe_forward_few, moe_linear and moe_linear_backward without a GPU: what
they refuse, before any launch, and their workspace sizes."""

import ctypes
from dataclasses import replace

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C

V3, TINY, FP4 = C.V3_PREFILL.cfg, C.TINY_FP32.cfg, C.V41_FLASH_FP4.cfg
OK, BAD, UNSUP, WS = B.MOE_OK, B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


def addr(i):
    return ctypes.c_void_p(0x100000 * (i + 1))


def few(cfg, T=4, x=addr(50), y=addr(51), ids=None, ws=addr(52), ws_bytes=1 << 40, **weights):
    w = B.MoeWeightsC(*[addr(i) for i in range(12)])
    for n, v in weights.items():
        setattr(w, n, v)
    return B._lib.moe_forward_few(ctypes.byref(B.config_c(cfg)), ctypes.byref(w), x, ids, T, y, ws,
                                  ws_bytes, None)


def test_few_refuses_before_any_launch():
    lib, cc = B._lib, B.config_c(V3)
    w = B.MoeWeightsC(*[addr(i) for i in range(12)])
    assert few(V3, T=-1) == BAD
    assert few(V3, T=17) == UNSUP
    assert few(replace(V3, dim=(1 << 20) + 64)) == UNSUP
    assert few(replace(V3, moe_inter_dim=(1 << 20) + 64)) == UNSUP
    assert few(replace(V3, dim=7168 + 32)) == UNSUP
    assert few(replace(V3, n_expert_groups=7)) == BAD
    assert lib.moe_forward_few(None, ctypes.byref(w), addr(0), None, 1, addr(1), addr(2), 1 << 40, None) == BAD
    assert lib.moe_forward_few(ctypes.byref(cc), None, addr(0), None, 1, addr(1), addr(2), 1 << 40, None) == BAD
    assert lib.moe_forward_few(ctypes.byref(cc), None, None, None, 0, None, None, 0, None) == BAD
    assert few(V3, x=None) == BAD and few(V3, y=None) == BAD and few(V3, x=addr(1), y=addr(1)) == BAD
    for n in ("w_gate", "w_up", "w_down", "gate_w", "sh_gate", "sh_up", "sh_down"):
        assert few(V3, **{n: None}) == BAD, n
        assert few(V3, **{n: ctypes.c_void_p(0x100008)}) == BAD, n
    assert few(V3, x=ctypes.c_void_p(0x100008)) == BAD
    assert few(V3, y=ctypes.c_void_p(0x100008)) == BAD
    assert few(FP4, s_up=None) == BAD
    assert few(C.HASH_BF16.cfg) == BAD                       # no ids
    assert few(C.HASH_BF16.cfg, ids=addr(60), tid2eid=None) == BAD
    assert few(C.NGRAM_BF16.cfg) == BAD
    size = B.moe_few_workspace_size(V3, 4)
    assert few(V3, ws=None) == WS
    assert few(V3, ws_bytes=size - 1) == WS
    assert few(V3, ws=ctypes.c_void_p(0x100080)) == WS
    assert few(V3, T=0, x=None, y=None, ws=None) == OK       # nothing to do


def test_few_workspace():
    assert B.moe_few_workspace_size(V3, 17) == 0
    assert B.moe_few_workspace_size(V3, -1) == 0
    last = 0
    for T in range(1, 17):
        lay = B.moe_few_workspace_layout(V3, T)
        assert lay["total_bytes"] == B.moe_few_workspace_size(V3, T) >= last
        last = lay["total_bytes"]
        parts = sorted(v for n, v in lay.items() if n not in ("total_bytes", "h_lo"))
        assert all(v % 256 == 0 for v in parts) and parts[0] == 0
    assert B.moe_few_workspace_size(C.V41_FLASH_FP4_MX.cfg, 16) > B.moe_few_workspace_size(FP4, 16)
    with pytest.raises(B.MoEError):
        B.alloc_few_workspace(V3, 17, "cpu")


def lin(M=8, K=64, N=32, dtype=1, act=0, limit=0.0, ld_x=0, ld_y=0, ld_r=0, x=addr(1), w=addr(2),
        w_up=None, bias=None, bias_up=None, res=None, y=addr(3), z=None, z_up=None, ws=addr(9),
        ws_bytes=1 << 40):
    c = B.MoeLinearConfigC(M, K, N, dtype, act, limit, ld_x, ld_y, ld_r)
    return B._lib.moe_linear(ctypes.byref(c), ctypes.byref(B.MoeLinearWeightsC(w, w_up, bias, bias_up)),
                             x, res, y, z, z_up, ws, ws_bytes, None)


ODD = ctypes.c_void_p(0x100008)
HALF = ctypes.c_void_p(0x100001)


@pytest.mark.parametrize("status,change", [
    (BAD, dict(M=-1)), (BAD, dict(K=0)), (BAD, dict(N=0)), (BAD, dict(dtype=2)), (BAD, dict(dtype=-1)),
    (BAD, dict(act=6)), (BAD, dict(act=-1)), (BAD, dict(limit=-1.0)), (BAD, dict(limit=float("nan"))),
    (BAD, dict(limit=float("inf"))), (BAD, dict(limit=1.0)),          # a clamp without swiglu
    (BAD, dict(ld_x=63)), (BAD, dict(ld_y=31)), (BAD, dict(ld_r=31)),
    (UNSUP, dict(ld_x=(1 << 20) + 8)), (UNSUP, dict(K=(1 << 20) + 8)), (UNSUP, dict(M=1 << 31)),
    (BAD, dict(x=None)), (BAD, dict(y=None)), (BAD, dict(w=None)), (BAD, dict(x=addr(3))),
    (BAD, dict(x=ODD)), (BAD, dict(w=ODD)), (BAD, dict(y=HALF)), (BAD, dict(bias=HALF)),
    (BAD, dict(res=HALF)), (BAD, dict(w_up=addr(4))), (BAD, dict(bias_up=addr(4))),
    (BAD, dict(act=5)), (BAD, dict(act=5, w_up=ODD)), (BAD, dict(act=5, w_up=addr(4), z=addr(5))),
    (BAD, dict(z_up=addr(5))), (BAD, dict(z=addr(5), z_up=addr(6))), (BAD, dict(y=addr(5), z=addr(5))),
    (BAD, dict(res=addr(3), ld_r=40)),                                # in place, other strides
    (WS, dict(K=63, ws=None)), (WS, dict(K=63, ws_bytes=16)), (WS, dict(K=63, ws=ctypes.c_void_p(0x180))),
    (OK, dict(M=0, x=None, y=None, ws=None)),
])
def test_linear_refuses_before_any_launch(status, change):
    assert lin(**change) == status


def back(M=8, K=64, N=32, act=0, x=addr(1), w=addr(2), w_up=None, dy=addr(3), z=None, z_up=None,
         ws=addr(9), ws_bytes=1 << 40, ld_y=0, grads=None, **g):
    c = B.MoeLinearConfigC(M, K, N, 1, act, 0.0, 0, ld_y, 0)
    gr = B.MoeLinearGradsC(*[g.get(n) for n in ("dx", "dw", "dw_up", "dbias", "dbias_up")])
    return B._lib.moe_linear_backward(
        ctypes.byref(c), ctypes.byref(B.MoeLinearWeightsC(w, w_up, None, None)), x, dy, z, z_up,
        None if grads == "null" else ctypes.byref(gr), ws, ws_bytes, None)


D = addr(20)


@pytest.mark.parametrize("status,change", [
    (BAD, dict()), (BAD, dict(grads="null")), (BAD, dict(dw_up=D)), (BAD, dict(dbias_up=D)),
    (BAD, dict(dx=D, dy=None)), (BAD, dict(dx=D, dy=ODD)), (BAD, dict(dx=D, w=None)),
    (BAD, dict(dw=D, x=None)), (BAD, dict(dw=D, x=ODD)), (BAD, dict(dx=D, w=ODD)),
    (BAD, dict(dx=D, act=2)), (BAD, dict(dx=D, act=5, z=addr(6), w_up=addr(7))),
    (BAD, dict(dx=D, act=5, z=addr(6), z_up=addr(8))), (BAD, dict(dx=addr(3))), (BAD, dict(dx=addr(1))),
    (BAD, dict(dw=HALF)), (BAD, dict(dbias=HALF)), (BAD, dict(dx=D, ld_y=31)),
    (WS, dict(dx=D, act=2, z=addr(6), ws=None)), (WS, dict(dbias=D, ws_bytes=8)),
])
def test_backward_refuses_before_any_launch(status, change):
    assert back(**change) == status


def test_linear_workspace_sizes():
    size = B.moe_linear_workspace_size
    c = C.LinearConfig(4096, 2048, 1024, "bf16", "swiglu")
    assert size(c) >= 256
    assert size(c, True) >= 2 * 4096 * 1024 * 2               # dz and du
    odd = C.LinearConfig(100, 63, 64)
    assert size(odd) >= 2 * 64 * (100 + 64)                   # padded copies of x and w
    assert size(C.LinearConfig(100, 64, 64), ld_x=67) >= 2 * 64 * 100
    assert size(C.LinearConfig(1, 0, 4)) == 0
    assert size(C.LinearConfig(0, 8, 8), True) >= 256
    with pytest.raises(B.MoEError):
        B.alloc_linear_workspace(C.LinearConfig(1, 0, 4), device="cpu")


def test_binding_checks_shapes_and_types():
    c = C.LinearConfig(4, 8, 16, "bf16", "none")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    x, w, y = bf(4, 8), bf(16, 8), bf(4, 16)
    for kw in (dict(x=bf(4, 9)), dict(x=x.float()), dict(w=bf(8, 16)), dict(y=bf(4, 8)),
               dict(w=bf(16, 16)[:, :8]), dict(x=bf(8, 4).t()), dict(bias=bf(8)),
               dict(residual=bf(16)), dict(z=bf(4, 32)[:, :16])):
        a = {"x": x, "w": w, "y": y, **kw}
        with pytest.raises(ValueError):
            B.moe_linear(c, a.pop("x"), a.pop("w"), a.pop("y"), stream=0, **a)
    with pytest.raises(ValueError):
        B.moe_linear_backward(c, y, x, w, dw=bf(8, 16), stream=0)
    with pytest.raises(ValueError):
        B.moe_linear_backward(c, y.float(), x, w, dw=w, stream=0)
