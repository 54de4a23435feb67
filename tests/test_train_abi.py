"""Rows to experts and back, 8-bit checkpoints and the experts' products without a
GPU: what they refuse, before any launch, and their workspace sizes."""

import ctypes
from dataclasses import replace

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C

OK, BAD, UNSUP, WS = B.MOE_OK, B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
CFG = C.MoEConfig(dim=64, n_routed_experts=8, n_activated_experts=2, moe_inter_dim=96)
BIG = 1 << 33


def at(i):
    return BIG * (i + 1)


def ref(cfg):
    return ctypes.byref(B.config_c(cfg))


def dispatch(cfg=CFG, T=4, R=8, x=at(1), inv=at(2), rows=at(3)):
    return B._lib.moe_dispatch(ref(cfg), x, inv, T, R, rows, None)


def combine(cfg=CFG, T=4, R=8, rows=at(1), inv=at(2), w=at(3), add=None, y=at(4)):
    return B._lib.moe_combine(ref(cfg), rows, inv, w, add, T, R, y, None)


def combine_back(cfg=CFG, T=4, R=8, dy=at(1), rows=at(2), inv=at(3), w=at(4), drows=at(5), dw=at(6)):
    return B._lib.moe_combine_backward(ref(cfg), dy, rows, inv, w, T, R, drows, dw, None)


def test_rows_refuse_before_any_launch():
    wide = replace(CFG, dim=1 << 20)
    for call in (dispatch, combine, combine_back):
        assert call(T=-1) == BAD and call(R=-1) == BAD
        assert call(replace(CFG, dim=0)) == BAD and call(replace(CFG, n_activated_experts=0)) == BAD
        assert call(replace(CFG, act_dtype="fp4")) == BAD
        assert call(replace(CFG, n_activated_experts=17)) == UNSUP
        assert call(T=1 << 30) == UNSUP                      # T k past 31 bits
        assert call(wide, T=1 << 16) == UNSUP                # 2^33 pieces of 16 bytes
        assert call(R=1 << 31) == UNSUP
        assert call(replace(CFG, dim=(1 << 31) - 1), T=1) == UNSUP
        assert call(inv=None) == BAD and call(inv=at(2) + 2) == BAD
        assert call(T=0) == OK
    assert dispatch(x=None) == BAD and dispatch(rows=None) == BAD
    assert dispatch(x=at(1) + 1) == BAD and dispatch(rows=at(3) + 1) == BAD
    assert dispatch(rows=at(1)) == BAD and dispatch(rows=at(1) + 64) == BAD   # inside x
    assert dispatch(rows=at(2) + 16) == BAD                  # over the indices
    assert dispatch(R=0, rows=None) == OK
    assert combine(rows=None) == BAD and combine(w=None) == BAD and combine(y=None) == BAD
    assert combine(y=at(1) + 128) == BAD and combine(add=at(4)) == BAD
    assert combine(w=at(3) + 2) == BAD and combine(add=at(5) + 1) == BAD
    assert combine_back(drows=None, dw=None) == BAD and combine_back(dy=None) == BAD
    assert combine_back(w=None) == BAD and combine_back(rows=None) == BAD
    assert combine_back(drows=at(1)) == BAD and combine_back(drows=at(2)) == BAD
    assert combine_back(dw=at(5) + 4) == BAD and combine_back(dw=at(4)) == BAD
    lib = B._lib.moe_dispatch_backward
    assert lib(ref(CFG), at(1), at(2), 4, 8, at(1), None) == BAD
    assert lib(ref(CFG), None, at(2), 4, 8, at(3), None) == BAD
    assert lib(None, at(1), at(2), 4, 8, at(3), None) == BAD


def save(src=at(1), dtype=1, rows=4, cols=40, ld=0, limit=0.0, codes=at(2), scales=at(3)):
    return B._lib.moe_checkpoint_save(src, dtype, rows, cols, ld, limit, codes, scales, None)


def load(codes=at(2), scales=at(3), dtype=1, rows=4, cols=40, ld=0, dst=at(1)):
    return B._lib.moe_checkpoint_load(codes, scales, dtype, rows, cols, ld, dst, None)


def test_checkpoints_refuse_before_any_launch():
    for call in (save, load):
        assert call(dtype=2) == BAD and call(rows=-1) == BAD and call(cols=0) == BAD
        assert call(ld=39) == BAD
        assert call(rows=1 << 31) == UNSUP and call(rows=1 << 28, cols=1 << 10) == UNSUP
        assert call(rows=1, cols=(1 << 31) - 1) == UNSUP and call(rows=1, cols=(1 << 31) - 31) == UNSUP
        assert call(codes=None) == BAD and call(scales=None) == BAD
        assert call(rows=0) == OK
    assert save(src=None) == BAD and load(dst=None) == BAD
    assert save(src=at(1) + 1) == BAD and save(dtype=0, src=at(1) + 2) == BAD
    for limit in (-1.0, float("inf"), float("nan")):
        assert save(limit=limit) == BAD
    assert save(codes=at(1) + 100) == BAD and save(codes=at(3) - 100) == BAD
    assert load(dst=at(2) + 150) == BAD


def weights(**change):
    w = B.MoeWeightsC()
    w.w_gate, w.w_up, w.w_down = at(10), at(11), at(12)
    for n, v in change.items():
        setattr(w, n, v)
    return w


def kept(kind=2, **change):
    s = B.MoeExpertsSavedC(kind, at(20), at(21), at(22), at(23))
    for n, v in change.items():
        setattr(s, n, v)
    return ctypes.byref(s)


def experts(cfg=CFG, rows=10, x=at(1), off=at(2), y=at(3), saved=None, ws=at(4), ws_bytes=1 << 30, w=None):
    return B._lib.moe_experts(ref(cfg), ctypes.byref(w or weights()), x, off, rows, y, saved, ws,
                              ws_bytes, None)


def back(cfg=CFG, rows=10, x=at(1), off=at(2), dy=at(3), saved=(), ws=at(4), ws_bytes=1 << 30, w=None, **g):
    grads = B.MoeExpertsGradsC(at(30), at(31), at(32), at(33))
    for n, v in g.items():
        setattr(grads, n, v)
    return B._lib.moe_experts_backward(ref(cfg), ctypes.byref(w or weights()), x, off, rows, dy,
                                       kept() if saved == () else saved, ctypes.byref(grads), ws,
                                       ws_bytes, None)


@pytest.mark.parametrize("call", [experts, back])
def test_experts_refuse_before_any_launch(call):
    assert call(rows=-1) == BAD and call(rows=1 << 31) == UNSUP
    assert call(replace(CFG, n_routed_experts=1), rows=(1 << 31) - 64) == UNSUP
    # offsets [0, rows, 0, rows, ..] would make more tiles than 31 bits count
    assert call(replace(CFG, n_routed_experts=1024), rows=1 << 29) == UNSUP
    for change in (dict(dim=0), dict(n_routed_experts=0), dict(moe_inter_dim=0),
                   dict(swiglu_limit=-1.0), dict(swiglu_limit=float("inf")),
                   dict(swiglu_limit=float("nan")), dict(act_dtype="fp8")):
        assert call(replace(CFG, **change)) == BAD, change
    for change in (dict(expert_dtype="fp4"), dict(act_dtype="f32"), dict(weight_layout="tiled"),
                   dict(act_quant="mxfp8"), dict(dim=68), dict(moe_inter_dim=100),
                   dict(n_routed_experts=1025), dict(dim=(1 << 20) + 8),
                   dict(moe_inter_dim=(1 << 20) + 8), dict(dim=1 << 20, moe_inter_dim=1 << 20,
                                                           n_routed_experts=1024)):
        assert call(replace(CFG, **change)) == UNSUP, change
    assert call(replace(CFG, moe_inter_dim=72), saved=kept()) == UNSUP     # no whole blocks of 32
    assert call(saved=kept(3)) == BAD and call(saved=kept(-1)) == BAD
    for n in ("gate", "up", "gate_scales", "up_scales"):
        assert call(saved=kept(**{n: None})) == BAD, n
    assert call(saved=kept(gate=at(20) + 8)) == BAD
    for n in ("w_gate", "w_up", "w_down"):
        assert call(w=weights(**{n: None})) == BAD, n
        assert call(w=weights(**{n: at(10) + 8})) == BAD, n
    assert call(off=None) == BAD and call(off=at(2) + 2) == BAD and call(x=None) == BAD
    assert call(x=at(1) + 8) == BAD
    size = B.moe_experts_workspace_size(CFG, 10, call is back)
    assert call(ws=None) == WS and call(ws=at(4) + 128) == WS and call(ws_bytes=size - 1) == WS
    assert call(ws=at(1) + 256) == BAD                       # inside x


@pytest.mark.parametrize("E,d,I", [(2, 64, 1 << 20), (4, 64, 1 << 20), (1024, 64, 1 << 20),
                                   (1024, 1 << 20, 64), (1, 64, 1 << 20), (7, 1 << 20, 64)])
def test_experts_tiles_can_be_counted(E, d, I):
    """Of the largest sizes that are taken the tiles stay below 2^31, whatever the offsets:
    expert after expert all rows and none, two neighbours with a block of 64 rows
    more than their rows make, and room for workgroups that step past the last."""
    cfg, lo, hi = replace(CFG, n_routed_experts=E, dim=d, moe_inter_dim=I), 0, 1 << 25
    while hi - lo > 1:                                       # blocks of 64 rows
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if B.moe_experts_workspace_size(cfg, 64 * mid) else (lo, mid)
    rows = 64 * lo
    assert lo > 100 and B.moe_experts_workspace_size(cfg, rows + 64) == 0
    offsets = [0] if E % 2 else [0, 1]
    while len(offsets) <= E:
        offsets.append(0 if offsets[-1] == rows else rows)
    blocks = sum(-(-max(b - a, 0) // 64) for a, b in zip(offsets, offsets[1:]))
    assert blocks * max(-(-d // 64), -(-I // 32)) < (1 << 31) - 1024


def test_experts_overlaps():
    assert experts(y=at(1)) == BAD and experts(y=at(1) + 64) == BAD and experts(y=at(12) + 16) == BAD
    assert experts(saved=kept(up=at(20) + 32)) == BAD        # z's codes run into u's
    assert experts(saved=kept(gate=at(1))) == BAD
    assert experts(y=None) == BAD
    assert experts(rows=0, x=None, y=None, off=None, ws=None) == OK
    assert back(dx=None, dw_gate=None, dw_up=None, dw_down=None) == BAD
    assert back(dy=None) == BAD and back(saved=None) == BAD and back(saved=kept(0)) == BAD
    assert back(dx=at(3)) == BAD and back(dx=at(1) + 64) == BAD and back(dw_down=at(12)) == BAD
    assert back(dw_up=at(31) + 128) == BAD and back(dx=at(21) + 16) == BAD
    assert back(dw_gate=at(31) + 8) == BAD and back(dy=at(3) + 8) == BAD


def test_gradients_of_nothing():
    """Outputs without elements have no address: a rank without tokens, or without a row,
    makes the same calls."""
    assert combine_back(T=0, R=0, drows=None, dw=None) == OK
    assert combine_back(T=0, dw=None) == OK and combine_back(T=0, R=0, dy=None, rows=None) == OK
    assert combine_back(R=0, rows=None, drows=None, dw=None) == OK
    assert combine_back(T=0, drows=None, dw=None, inv=None, w=None) == OK
    assert combine_back(T=-1, drows=None, dw=None) == BAD
    none, inv, w = bf(0, 64), torch.zeros((0, 2), dtype=torch.int32), torch.zeros((0, 2))
    B.moe_combine_backward(CFG, none, none, inv, w, 0, drows=none.clone(), dweights=w.clone(), stream=0)
    assert back(rows=0, dx=None, dw_gate=None, dw_up=None, dw_down=None) == OK
    assert back(rows=0, off=None, dx=None, dw_gate=None, dw_up=None, dw_down=None) == BAD


def test_experts_workspace():
    one = B.moe_experts_workspace_size(CFG, 1000)
    assert one >= 1000 * 96 * 2 and one % 256 == 0
    assert B.moe_experts_workspace_size(CFG, 1000, True) >= 3 * 1000 * 96 * 2
    assert B.moe_experts_workspace_size(CFG, 0) == 256
    assert B.moe_experts_workspace_size(replace(CFG, dim=68), 10) == 0
    assert B.alloc_experts_workspace(CFG, 10, True, "cpu").numel() >= 3 * 10 * 96 * 2
    with pytest.raises(B.MoEError):
        B.alloc_experts_workspace(replace(CFG, dim=68), 10, True, "cpu")
    s = B.alloc_experts_saved(CFG, 10, "mxfp8", "cpu")
    assert s["gate"].shape == (10, 96) and s["up_scales"].shape == (10, 3)
    assert B.alloc_experts_saved(CFG, 10, "full", "cpu")["up"].dtype is torch.float32
    with pytest.raises(ValueError):
        B.alloc_experts_saved(CFG, 10, "fp8", "cpu")


def bf(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses():
    inv, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    cases = [
        (B.moe_dispatch, (bf(4, 64), inv, 4, bf(8, 64)), "expected a GPU"),
        (B.moe_dispatch, (bf(4, 63), inv, 4, bf(8, 64)), "x is"),
        (B.moe_dispatch, (bf(4, 64), inv.long(), 4, bf(8, 64)), "inverse is"),
        (B.moe_dispatch, (bf(4, 64), inv, 4, bf(8, 128)[:, :64]), "not contiguous"),
        (B.moe_dispatch, (bf(4, 64), inv, 5, bf(8, 64)), "x is"),
        (B.moe_dispatch_backward, (bf(8, 64), inv, 4, bf(4, 64).to("meta")), "is on"),
        (B.moe_dispatch_backward, (bf(8, 64, dtype=torch.float32), inv, 4, bf(4, 64)), "drows is"),
        (B.moe_combine, (bf(8, 64), inv, w.double(), 4, bf(4, 64)), "weights is"),
        (B.moe_combine, (bf(8, 64), inv, w, 4, bf(4, 64)), "expected a GPU"),
        (B.moe_combine_backward, (bf(4, 64), bf(8, 64), inv, w, 4, bf(9, 64)), "drows is"),
    ]
    for call, args, message in cases:
        with pytest.raises(ValueError, match=message):
            call(CFG, *args, stream=0)
    with pytest.raises(ValueError, match="add is"):
        B.moe_combine(CFG, bf(8, 64), inv, w, 4, bf(4, 64), add=bf(4, 32), stream=0)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    for src, codes, scales, message in (
            (bf(4, 40), u8(4, 40), u8(4, 1), "scales is"),
            (bf(4, 40), u8(4, 41), u8(4, 2), "codes is"),
            (bf(4, 40).half(), u8(4, 40), u8(4, 2), "expected a matrix"),
            (bf(40, 4).t(), u8(4, 40), u8(4, 2), "rows are not contiguous"),
            (bf(1, 40).expand(4, 40), u8(4, 40), u8(4, 2), "overlap"),
            (bf(4, 40), u8(4, 40).to("meta"), u8(4, 2), "is on"),
            (bf(4, 40), u8(4, 40), u8(4, 2), "expected a GPU")):
        with pytest.raises(ValueError, match=message):
            B.moe_checkpoint_save(src, codes, scales, stream=0)
        with pytest.raises(ValueError, match=message):
            B.moe_checkpoint_load(codes, scales, src, stream=0)
    layer = {"w_gate": bf(8, 96, 64), "w_up": bf(8, 96, 64), "w_down": bf(8, 64, 96)}
    off, ws = torch.zeros(9, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    saved = B.alloc_experts_saved(CFG, 5, "mxfp8", "cpu")
    for change, message in (
            (dict(), "expected a GPU"), (dict(offsets=off[:8]), "offsets is"),
            (dict(y=bf(6, 64)), "y is"), (dict(layer={**layer, "w_up": bf(8, 64, 96)}), "w_up is"),
            (dict(saved={**saved, "gate": u8(5, 64)}), "gate is"),
            (dict(saved={**saved, "up_scales": u8(4, 3)}), "up_scales is"),
            (dict(ws=ws[::2]), "ws is not contiguous")):
        a = dict(layer=layer, x=bf(5, 64), offsets=off, y=bf(5, 64), ws=ws, saved=saved, stream=0)
        a.update(change)
        with pytest.raises(ValueError, match=message):
            B.moe_experts(CFG, **a)
    for grads, message in (({"dx": bf(5, 32)}, "dx is"), ({"dw_up": bf(8, 64, 96)}, "dw_up is"),
                           ({"w_up": bf(8, 96, 64)}, "grads has"), ({"dx": bf(5, 64)}, "a GPU")):
        with pytest.raises(ValueError, match=message):
            B.moe_experts_backward(CFG, layer, bf(5, 64), off, bf(5, 64), saved, grads, ws, stream=0)
