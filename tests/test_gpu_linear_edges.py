"""moe_linear and its gradient at their edges: slopes of very large
pre-activations, saved values around the clamp, addresses inside odd rows."""

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C
from tests import test_gpu_linear as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(8, 64), (2048, 1024)])       # the small and the tiled backward
@pytest.mark.parametrize("activation", ["gelu_tanh", "gelu", "silu"])
def test_slopes_of_large_values(activation, M, N, dtype, gpu):
    """1 and 0 far out, also where z^2 is past the largest float: through an
    identity dx is dz, and dbias its sum."""
    dt = L.DT[dtype]
    row = torch.tensor([1e3, 1e9, 1e13, 1.8e19, 2e19, 1e20, 1e30, 3e38], device=gpu)
    z = torch.cat([row, -row]).repeat(N // 16).expand(M, N).to(dt).contiguous()
    dy = torch.ones((M, N), dtype=dt, device=gpu)
    eye = torch.eye(N, dtype=dt, device=gpu)
    c = C.LinearConfig(M, N, N, dtype, activation)
    dx, db = torch.empty_like(dy), torch.empty(N, dtype=dt, device=gpu)
    B.moe_linear_backward(c, dy, dy, eye, z=z, dx=dx, dbias=db, ws=B.alloc_linear_workspace(c, True))
    torch.cuda.synchronize()
    assert torch.equal(dx, (z > 0).to(dt))
    assert torch.equal(db, (z[0] > 0).to(dt) * M)


@pytest.mark.parametrize("limit", [1.0, 0.7, 3.3])
def test_saved_gate_is_the_nearest_value_below_zero(limit, gpu):
    """The gate is clamped from above alone: around -L its saved value is the
    nearest one, as everywhere but at +L (sums of two terms, exact)."""
    steps = torch.arange(-40, 41, device="cuda").float() * 2.0 ** -10
    want = -limit + steps * limit
    hi = want.to(torch.bfloat16)
    lo = (want - hi.float()).to(torch.bfloat16)
    exact = hi.float() + lo.float()
    M = want.numel()
    x = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = hi, lo
    w = torch.zeros((8, 8), dtype=torch.bfloat16, device="cuda")
    w[:, 0] = w[:, 1] = 1
    c = C.LinearConfig(M, 8, 8, "bf16", "swiglu", limit)
    y, z, zu = L.outputs(c, {})
    B.moe_linear(c, x, w, y, w_up=w, z=z, z_up=zu, ws=B.alloc_linear_workspace(c))
    torch.cuda.synchronize()
    assert torch.equal(z[:, 0], exact.to(torch.bfloat16))
    bound = float(torch.tensor(limit, dtype=torch.float32))
    assert torch.equal(zu[:, 0].float() < -bound, exact < -bound)      # the up value has that border


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(1, 63, 5), (9, 777, 1023), (203, 63, 97), (2300, 515, 1031)])
@pytest.mark.parametrize("activation", ["none", "swiglu"])
def test_addresses_inside_odd_rows(M, K, N, activation, dtype, gpu):
    """x, dy and the weights from the second row or matrix of a larger one of
    odd widths, where no address is a multiple of 16 bytes."""
    c, t = L.make(M, K, N, dtype, activation, 31)
    for n in ("x", "dy", "w", "w_up"):
        if n in t:
            whole = torch.zeros((t[n].shape[0] + 1, t[n].shape[1]), dtype=t[n].dtype, device=gpu)
            whole[1:] = t[n]
            t[n] = whole[1:]
            assert t[n].data_ptr() % 16
    L.check_all(c, t, f"{dtype} {activation} {M}x{K}x{N} inside")
