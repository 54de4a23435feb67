"""Every kernel of the tiled dense product against float64: each tile shape of the
forward, of swiglu's, of dx (swiglu: two segments) and of dW (swiglu: two halves),
whole and with the contraction split, at ragged sizes, an active clamp among
them.  A case names the kernels that its sizes select, so that a change of the
choice cannot take one out of the tests unseen."""

import pytest

from mixture_experts_ffn_route_amd import binding as B
from tests import test_gpu_linear as L

pytestmark = pytest.mark.gpu

# dtype, activation, limit, rows, in, out: tiles of the forward, dx and dW ("/": split contraction)
CASES = [
    # gate|up widths of the named hash-routed and FP4 workloads in training
    ("bf16", "swiglu", 1.0, 4096, 2048, 1024, "256x128", "256x128", "128x128"),
    ("bf16", "swiglu", 1.5, 8192, 5120, 1536, "256x256", "256x256", "256x256"),
    # the smallest sizes that reach every kernel there is
    ("bf16", "silu", 0.0, 66, 64, 1168, "64x64", "64x64", "64x64"),
    ("bf16", "silu", 0.0, 1763, 1736, 71, "64x64/", "128x128", "64x64/"),
    ("bf16", "silu", 0.0, 226, 193, 8354, "128x128", "64x64/", "128x128"),
    ("bf16", "silu", 0.0, 5194, 2313, 68, "128x128/", "256x256", "128x128/"),
    ("bf16", "silu", 0.0, 1937, 604, 6621, "256x256", "128x128/", "256x128"),
    ("bf16", "silu", 0.0, 1227, 3288, 3752, "256x128", "256x128", "256x256"),
    ("bf16", "silu", 0.0, 421, 5873, 8356, "256x256/", "128x128", "256x256"),
    ("bf16", "silu", 0.0, 8444, 392, 6616, "256x256", "256x256/", "128x128"),
    ("bf16", "silu", 0.0, 6279, 4099, 908, "256x128", "256x256", "256x256/"),
    ("bf16", "swiglu", 1.0, 66, 64, 296, "64x128", "64x64", "64x64"),
    ("bf16", "swiglu", 1.0, 65, 1864, 834, "64x128/", "64x64/", "128x128"),
    ("bf16", "swiglu", 1.0, 2147, 2677, 65, "128x128/", "128x128", "64x64/"),
    ("bf16", "swiglu", 1.0, 149, 904, 6240, "128x128", "128x128/", "256x256"),
    ("bf16", "swiglu", 1.5, 6578, 600, 984, "256x256", "256x128", "128x128/"),
    ("bf16", "swiglu", 1.0, 4329, 3065, 650, "256x128", "256x256", "256x128"),
    ("bf16", "swiglu", 1.5, 8366, 160, 8464, "64x128", "256x256/", "256x256/"),
    ("bf16", "swiglu", 1.5, 5498, 6192, 336, "256x256/", "128x128", "256x128"),
    ("f32", "silu", 0.0, 67, 64, 1632, "64x64", "64x64/", "64x64"),
    ("f32", "silu", 0.0, 541, 2128, 64, "64x64/", "64x64", "64x64/"),
    ("f32", "silu", 0.0, 75, 3115, 6321, "128x128/", "128x128/", "128x128"),
    ("f32", "silu", 0.0, 6051, 632, 608, "128x128", "128x128", "128x128/"),
    ("f32", "swiglu", 1.0, 66, 64, 548, "64x128", "64x64/", "64x64"),
    ("f32", "swiglu", 1.0, 568, 1088, 69, "64x128/", "64x64", "64x64/"),
    ("f32", "swiglu", 1.5, 65, 3080, 3120, "128x128/", "128x128/", "128x128"),
    ("f32", "swiglu", 1.0, 5194, 594, 314, "128x128", "128x128", "128x128/"),
]


def tiles(c, t, product):
    path, rows, cols, parts = B.moe_linear_path(c, product, t["x"].stride(0), t["dy"].stride(0))
    return f"{rows}x{cols}" + ("/" if parts > 1 else "") if path == "tiled" else path


@pytest.mark.parametrize("dtype,activation,limit,M,K,N,forward,dx,dw", CASES)
def test_every_tile(dtype, activation, limit, M, K, N, forward, dx, dw, gpu):
    c, t = L.make(M, K, N, dtype, activation, 41, limit=limit)
    assert [tiles(c, t, p) for p in ("forward", "dx", "dw")] == [forward, dx, dw]
    L.check_all(c, t, f"{dtype} {activation} {limit} {M}x{K}x{N}")
