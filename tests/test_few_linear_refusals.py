"""What moe_forward_few, moe_linear and moe_linear_backward take and refuse,
without a GPU: nothing here comes to a launch."""

from dataclasses import replace

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C


@pytest.mark.parametrize("E,G,kept", [(48, 4, 2), (48, 8, 4), (96, 8, 4), (130, 65, 4), (504, 7, 3), (24, 24, 9)])
def test_few_takes_groups_of_any_size(E, G, kept):
    cfg = replace(C.V3_PREFILL.cfg, n_routed_experts=E, n_expert_groups=G, n_limited_groups=kept,
                  n_activated_experts=4)
    assert B.alloc_few_workspace(cfg, 16, "cpu").numel() == B.moe_few_workspace_size(cfg, 16) > 0
    with pytest.raises(B.MoEError):
        B.alloc_few_workspace(replace(cfg, n_limited_groups=G + 1), 16, "cpu")
    with pytest.raises(B.MoEError):
        B.alloc_few_workspace(replace(cfg, n_expert_groups=E - 1), 16, "cpu")


LINEAR = C.LinearConfig(4, 16, 8)


def bf(*shape, device="cpu"):
    return torch.zeros(shape, dtype=torch.bfloat16, device=device)


@pytest.mark.parametrize("grads", [dict(dw=bf(8, 16)), dict(dbias=bf(8)), dict(dw=bf(8, 16), dbias=bf(8))])
def test_empty_batch_has_its_gradients_checked(grads):
    """No rows: zeros are written all the same, so not to host memory."""
    c = replace(LINEAR, rows=0)
    with pytest.raises(ValueError, match="expected a GPU"):
        B.moe_linear_backward(c, bf(0, 8), bf(0, 16), bf(8, 16), stream=0, **grads)
    with pytest.raises(ValueError, match="expected a GPU"):
        B.moe_linear_backward(c, None, None, None, stream=0, **grads)
    with pytest.raises(ValueError, match="is on"):
        B.moe_linear_backward(c, bf(0, 8, device="meta"), None, None, stream=0, **grads)


def test_empty_forward_is_a_no_op():
    B.moe_linear(replace(LINEAR, rows=0), bf(0, 16), bf(8, 16), bf(0, 8), stream=0)


WRONG_WORKSPACES = [
    (torch.empty(4096, dtype=torch.uint8), "ws is on cpu"),
    (torch.empty((64, 64), dtype=torch.uint8, device="meta")[:, :32], "ws is not contiguous"),
]


@pytest.mark.parametrize("ws,message", WRONG_WORKSPACES)
def test_linear_checks_its_workspace(ws, message):
    """Tensors that are elsewhere than the workspace; the workspace in pieces."""
    x, w, y = (bf(*s, device="meta") for s in ((4, 16), (8, 16), (4, 8)))
    with pytest.raises(ValueError, match=message):
        B.moe_linear(LINEAR, x, w, y, ws=ws, stream=0)
    with pytest.raises(ValueError, match=message):
        B.moe_linear_backward(LINEAR, y, x, w, dx=x, ws=ws, stream=0)


FEW = replace(C.SMALL_WORKLOADS["hash_small"].cfg, dim=64, moe_inter_dim=64, n_routed_experts=4,
              n_activated_experts=2, vocab_size=10)


def few_layer(device):
    layer = {n: bf(4, 64, 64, device=device) for n in ("w_gate", "w_up", "w_down")}
    layer.update({n: bf(64, 64, device=device) for n in ("sh_gate", "sh_up", "sh_down")})
    layer["tid2eid"] = torch.zeros((10, 2), dtype=torch.int32, device=device)
    return layer


IDS = torch.zeros(3, dtype=torch.int32, device="meta")


@pytest.mark.parametrize("change,message", [
    (dict(x=bf(3, 63, device="meta")), "x holds"), (dict(x=bf(2, 64, device="meta")), "x holds"),
    (dict(x=bf(3, 64, device="meta").float()), "x is"), (dict(x=bf(64, 3, device="meta").t()), "x is not contiguous"),
    (dict(y=bf(2, 64, device="meta")), "y holds"), (dict(y=bf(3, 128, device="meta")[:, :64]), "y is not contiguous"),
    (dict(y=bf(3, 64)), "y is on cpu"), (dict(token_ids=torch.zeros(3, dtype=torch.int32)), "token_ids is on cpu"),
    (dict(token_ids=IDS.long()), "token_ids is"), (dict(token_ids=IDS[:2]), "token_ids holds"),
    (dict(ws=torch.empty(1 << 20, dtype=torch.uint8)), "ws is on cpu"),
    (dict(layer=few_layer("cpu")), "w_gate is on cpu"),
    (dict(layer=dict(few_layer("meta"), w_up=bf(4, 64, 128, device="meta")[..., :64])), "w_up is not contiguous"),
    (dict(), "expected a GPU"),
])
def test_few_checks_its_tensors(change, message):
    t = dict(x=bf(3, 64, device="meta"), y=bf(3, 64, device="meta"), token_ids=IDS,
             layer=few_layer("meta"), ws=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
    t.update(change)
    for cfg in (FEW, B.config_c(FEW)):
        with pytest.raises(ValueError, match=message):
            B.moe_forward_few(cfg, t["layer"], t["x"], t["token_ids"], 3, t["y"], t["ws"], stream=0)


def test_few_of_no_tokens_is_a_no_op():
    B.moe_forward_few(FEW, few_layer("cpu"), None, None, 0, None, None, stream=0)
    with pytest.raises(B.MoEError):
        B.moe_forward_few(FEW, few_layer("cpu"), None, None, -1, None, None, stream=0)


def status(M, K, N, dtype, x=0x1000, w=0x2000, ld_x=0, dy=0x3000, ld_y=0):
    """Of a forward and a backward call without a workspace: where the addresses
    pass, the workspace is what is missing."""
    c = B.MoeLinearConfigC(M, K, N, C.DTYPE[dtype], C.ACTIVATION["silu"], 0.0, ld_x, ld_y, 0)
    weights = B.MoeLinearWeightsC(w, None, None, None)
    grads = B.MoeLinearGradsC(0x5000, 0x6000)
    return (B._lib.moe_linear(c, weights, x, None, 0x4000, None, None, None, 0, None),
            B._lib.moe_linear_backward(c, weights, x, dy, 0x7000, None, grads, None, 0, None))


@pytest.mark.parametrize("dtype,size,whole", [("bf16", 2, 8), ("f32", 4, 4)])
def test_addresses_of_odd_rows(dtype, size, whole):
    """An element's alignment where rows are not whole 16-byte pieces, 16 bytes
    where they are; never less than an element's."""
    bad, ok = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_WORKSPACE
    K, N = 8 * whole + 1, 4 * whole + 1
    for change in (dict(x=0x1000 + size), dict(w=0x2000 + size)):
        assert status(8, K, N, dtype, **change) == (ok, ok)
    assert status(8, K, N, dtype, dy=0x3000 + size) == (ok, ok)
    assert status(8, 8 * whole, N, dtype, x=0x1000 + size, ld_x=9 * whole + 1) == (ok, ok)
    assert status(8, 8 * whole, N, dtype, x=0x1000 + size) == (bad, bad)
    assert status(8, 8 * whole, N, dtype, w=0x2000 + size, ld_x=9 * whole + 1) == (bad, bad)
    assert status(8, K, 4 * whole, dtype, dy=0x3000 + size) == (ok, bad)
    assert status(8, K, 4 * whole, dtype, dy=0x3000 + size, ld_y=5 * whole + 1) == (ok, ok)
    for change in (dict(x=0x1001), dict(w=0x2001)):
        assert status(8, K, N, dtype, **change) == (bad, bad)
    assert status(8, K, N, dtype, dy=0x3001) == (ok, bad)


def test_linear_path():
    c = C.LinearConfig(4096, 4096, 4096)
    assert B.moe_linear_path(c) == ("tiled", 256, 256, 1)
    assert B.moe_linear_path(replace(c, rows=16)) == ("few", 0, 0, 0)
    assert B.moe_linear_path(replace(c, rows=16), ld_x=4097)[0] != "few"
    small = C.LinearConfig(301, 256, 320, "f32", "silu")
    assert [B.moe_linear_path(small, p) for p in ("forward", "dx", "dw")] == [("small", 0, 0, 0)] * 3
    assert B.moe_linear_path(replace(c, rows=64, in_dim=8192, out_dim=72))[3] > 1
    for bad in (replace(c, in_dim=0), replace(c, rows=-1)):
        with pytest.raises(B.MoEError):
            B.moe_linear_path(bad)
    ok = B.MoeLinearConfigC(8, 8, 8, 1, 0, 0.0, 0, 0, 0)
    info = B.MoeLinearPathC()
    assert B._lib.moe_linear_path(ok, 3, info) == B._lib.moe_linear_path(ok, -1, info) == B.MOE_ERR_INVALID_ARG
    assert B._lib.moe_linear_path(ok, 0, None) == B._lib.moe_linear_path(None, 0, info) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("M,K,N,fits", [
    (1 << 20, 8192, 8192, (True, True)), (1 << 29, 64, 8, (True, True)), ((1 << 31) - 1, 8, 8, (False, False)),
    ((1 << 30) - 1024, 8, 8, (True, True)), (1 << 30, 8, 8, (False, False)), (1 << 30, 33, 8, (False, False)),
    (64, (1 << 20) - 1, (1 << 20) - 1, (False, False))])
def test_sizes_past_a_launch(M, K, N, fits):
    """Refused before anything is launched where a launch would have 2^32 threads."""
    c = C.LinearConfig(M, K, N)
    assert tuple(B.moe_linear_workspace_size(c, back) > 0 for back in (False, True)) == fits
    want = tuple(B.MOE_ERR_UNSUPPORTED if not f else None for f in fits)
    got = status(M, K, N, "bf16")
    assert all(w in (None, g) for g, w in zip(got, want)) and not any(
        w is None and g == B.MOE_ERR_UNSUPPORTED for g, w in zip(got, want))
