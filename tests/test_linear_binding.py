"""What the dense product's Python entry points refuse before the library sees
an address."""

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C

CFG = C.LinearConfig(4, 16, 8)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("change,message", [
    (dict(x=bf(1, 16).expand(4, 16)), "overlap"),             # every row the same memory
    (dict(x=bf(16, 4).t()), "rows are not contiguous"),
    (dict(residual=bf(8).expand(4, 8)), "overlap"),
    (dict(y=bf(4, 16)[:, ::2]), "rows are not contiguous"),
    (dict(w=bf(8, 24)[:, :16]), "not contiguous"),
    (dict(bias=bf(16)[::2]), "not contiguous"),
    (dict(x=bf(4, 16).to("meta")), "is on"),                  # tensors on two devices
    (dict(bias=bf(8).to("meta")), "is on"),
    (dict(), "expected a GPU"),                               # host memory
])
def test_forward_refuses(change, message):
    t = dict(x=bf(4, 16), w=bf(8, 16), y=bf(4, 8))
    t.update(change)
    with pytest.raises(ValueError, match=message):
        B.moe_linear(CFG, t.pop("x"), t.pop("w"), t.pop("y"), stream=0, **t)


@pytest.mark.parametrize("change,message", [
    (dict(dy=torch.ones((), dtype=torch.bfloat16).expand(4, 8)), "rows are not contiguous"),
    (dict(dy=bf(1, 8).expand(4, 8)), "overlap"),
    (dict(dx=bf(1, 16).expand(4, 16)), "overlap"),
    (dict(dw=bf(8, 32)[:, :16]), "not contiguous"),
    (dict(dw=bf(8, 16)), "expected a GPU"),
])
def test_backward_refuses(change, message):
    t = dict(dy=bf(4, 8), x=bf(4, 16), w=bf(8, 16))
    t.update(change)
    with pytest.raises(ValueError, match=message):
        B.moe_linear_backward(CFG, t.pop("dy"), t.pop("x"), t.pop("w"), stream=0, **t)


@pytest.mark.parametrize("K,N,dtype", [(64, 32, "bf16"), (63, 32, "bf16"), (4096, 1024, "f32")])
def test_a_workspace_without_strides_serves_all(K, N, dtype):
    c = C.LinearConfig(3000, K, N, dtype)
    n = B.alloc_linear_workspace(c, True, "cpu").numel()
    for back in (False, True):
        for ld_x in (0, K + 1, K + 2, K + 8):
            for ld_y in (0, N + 1, N + 4, N + 8):
                assert B.moe_linear_workspace_size(c, back, ld_x=ld_x, ld_y=ld_y) <= n


def test_outputs_are_not_inputs():
    """Addresses that an output and an input, or two outputs, share."""
    import ctypes
    p = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(8)]
    c = B.MoeLinearConfigC(8, 64, 64, 1, 0, 0.0, 0, 0, 0)
    w = B.MoeLinearWeightsC(p[1], None, p[2], None)

    def forward(y, z=None, residual=None):
        return B._lib.moe_linear(ctypes.byref(c), ctypes.byref(w), p[0], residual, y, z, None, None, 0, None)

    for out in (p[0], p[1], p[2]):
        assert forward(out) == B.MOE_ERR_INVALID_ARG
        assert forward(p[3], out) == B.MOE_ERR_INVALID_ARG
    assert forward(p[3], p[3]) == B.MOE_ERR_INVALID_ARG
    assert forward(p[3], p[4], p[4]) == B.MOE_ERR_INVALID_ARG

    s = B.MoeLinearConfigC(8, 64, 64, 1, 2, 0.0, 0, 0, 0)

    def backward(**g):
        gr = B.MoeLinearGradsC(*[g.get(n) for n in ("dx", "dw", "dw_up", "dbias", "dbias_up")])
        return B._lib.moe_linear_backward(ctypes.byref(s), ctypes.byref(w), p[0], p[3], p[4], None,
                                          ctypes.byref(gr), None, 0, None)

    for name in ("dx", "dw", "dbias"):
        for taken in (p[0], p[1], p[3], p[4]):
            assert backward(**{name: taken}) == B.MOE_ERR_INVALID_ARG
    assert backward(dx=p[6], dw=p[6]) == B.MOE_ERR_INVALID_ARG


def test_dx_stride_checks():
    import ctypes
    p = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(8)]
    c = B.MoeLinearConfigC(8, 64, 64, 1, 0, 0.0, 0, 0, 0)
    w = B.MoeLinearWeightsC(p[1], None, None, None)
    for ld, status in ((63, B.MOE_ERR_INVALID_ARG), (-1, B.MOE_ERR_INVALID_ARG),
                       ((1 << 20) + 1, B.MOE_ERR_UNSUPPORTED)):
        gr = B.MoeLinearGradsC(p[6], None, None, None, None, ld)
        assert B._lib.moe_linear_backward(ctypes.byref(c), ctypes.byref(w), None, p[3], None, None,
                                          ctypes.byref(gr), None, 0, None) == status
