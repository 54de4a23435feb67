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
