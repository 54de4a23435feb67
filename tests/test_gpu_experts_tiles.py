"""Every tile shape of the experts' products on the GPU, each case asserting the
shapes that it is there for: all heights of the largest tiles, streamed weights, last
rounds cut lower, tiles that workgroups walk one after another."""

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from tests import train_helpers as H
from tests.test_gpu_experts import GRADS, Step

pytestmark = pytest.mark.gpu

LARGE, STREAMED, MIDDLE, SMALL = (256, 256, False), (256, 256, True), (128, 128, False), (64, 64, False)
FLAT = (64, 256, False)
FEW = [(i * 5) % 9 for i in range(62)] + [130, 65]
MANY = [(i * 37) % 90 for i in range(66)] + [330, 256, 257, 193]

CASES = [
    # every height, most experts with little; 210 to 1050 tiles on 256 CUs
    (MANY, 520, 544, dict(up=LARGE, down=LARGE, dh=STREAMED, dx=STREAMED, dw_down=LARGE, dw=LARGE)),
    # a few rows an expert: 64 x 256, 320 and more tiles; two experts with several
    (FEW, 1032, 544, dict(up=FLAT, down=FLAT, dh=MIDDLE)),
    # one expert: weights read by five row tiles; 275 tiles, the last rounds cut in four
    ([1100], 14080, 32, dict(down=LARGE, dx=LARGE, up=(64, 128, False))),
    ([1100], 32, 14080, dict(up=LARGE, dh=LARGE, down=SMALL)),
    # 128 x 128, 528 tiles on 512 places, the last round cut in two
    ([1000], 8448, 64, dict(down=MIDDLE, dx=MIDDLE)),
    ([1000], 64, 8448, dict(up=MIDDLE, dh=MIDDLE)),
    ([1000], 64, 4736, dict(up=MIDDLE, dh=MIDDLE)),
    ([40, 0, 7, 100, 65, 1, 0, 33], 512, 1024, dict(dw_down=MIDDLE, dw=MIDDLE)),
    # heights of the gradients' tiles that do not divide: 5, 6 and 7 blocks
    ([3, 70, 0, 31] * 25, 424, 352, dict(dw_down=LARGE, dw=LARGE)),
]


@pytest.mark.parametrize("kind", ["mxfp8", "full"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tiles(gpu, case, kind):
    counts, d, I, paths = CASES[case]
    print(f"[tiles] rows={sum(counts)} E={len(counts)} d={d} I={I} {kind}", flush=True)
    s = Step(counts, d, I, "bf16", spare=3, limit=1.5 if case % 2 else 0.0).to(gpu, kind)
    for product, path in paths.items():
        assert B.moe_experts_path(s.cfg, s.rows, product) == path, product
    s.forward()
    s.check_forward()
    s.backward()
    s.check_backward()
    # the same again, with the workspace as the first pass left it
    first = [s.y.clone()] + [s.grads[n].clone() for n in GRADS]
    s.forward()
    s.backward()
    assert all(torch.equal(a, b) for a, b in zip(first, [s.y] + [s.grads[n] for n in GRADS]))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_tiles_without_saving(gpu, case):
    """Nothing saved: kernels of their own for every tile of up, the same y."""
    counts, d, I, paths = CASES[case]
    print(f"[tiles] rows={sum(counts)} E={len(counts)} d={d} I={I} none", flush=True)
    s = Step(counts, d, I, "bf16", spare=3, limit=1.5 if case % 2 else 0.0).to(gpu, "full")
    s.forward()
    s.check_forward()
    want = s.y.clone()
    s.kind = "none"
    s.y.fill_(-7.0)
    s.ws.fill_(0xFF)
    s.forward()
    assert torch.equal(s.y, want)


def test_1024_experts(gpu):
    """More experts than lanes: each lane scans sixteen."""
    counts = [(i * 7) % 5 if i % 3 else 0 for i in range(1024)]
    s = Step(counts, 16, 32, "bf16").to(gpu, "mxfp8")
    s.forward()
    s.backward()
    y, dx = s.y.cpu(), s.grads["dx"].cpu()
    dw = {n: s.grads[n].cpu() for n in GRADS[1:]}
    for e in (0, 1, 2, 16, 17, 511, 512, 700, 1021, 1022, 1023):
        part, w = s.expert(e)
        if counts[e] == 0:
            assert all((dw[n][e] == 0).all() for n in dw)
            continue
        H.check(f"y of expert {e}", y[part], *H.experts_forward(s.x[part], *w, 0.0)["y"])
        want = H.experts_backward(s.x[part], *w, *s.kept(part), s.dy[part], 0.0)
        H.check(f"dx of expert {e}", dx[part], *want["dx"])
        for n in dw:
            H.check(f"{n} of expert {e}", dw[n][e], *want[n])


def test_rows_past_32_bits(gpu):
    """Sorted rows whose elements and bytes pass 32 bits: an expert at the end of the
    buffer, and one that starts past the border."""
    d, I, rows = 4096, 32, 1_100_000                          # 4.5e9 elements of x
    n = [5, rows - 5 - 70, 70]
    s = Step([5, 0, 70], d, I, "bf16", seed=3)
    cfg = s.cfg
    layer = {k: v.to(gpu) for k, v in s.layer.items()}
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device=gpu)
    y = torch.zeros_like(x)
    x[:5], x[-70:] = s.x[:5].to(gpu), s.x[5:].to(gpu)
    off = torch.tensor([0, n[0], n[0] + n[1], rows], dtype=torch.int32, device=gpu)
    ws = B.alloc_experts_workspace(cfg, rows, True, gpu)
    saved = B.alloc_experts_saved(cfg, rows, "mxfp8", gpu)
    B.moe_experts(cfg, layer, x, off, y, ws, saved=saved)
    for e, part, mine in ((0, slice(0, 5), slice(0, 5)), (2, slice(5, 75), slice(rows - 70, rows))):
        w = s.expert(e)[1]
        H.check(f"y of expert {e}", y[mine], *H.experts_forward(s.x[part], *w, 0.0)["y"])
    assert (y[5:-70] == 0).all()
    dy, dx = y, x                                             # dx in place of another buffer is refused
    with pytest.raises(B.MoEError):
        B.moe_experts_backward(cfg, layer, x, off, dy, saved, {"dx": dx}, ws)
    dx = torch.zeros_like(x)
    B.moe_experts_backward(cfg, layer, None, off, dy, saved, {"dx": dx}, ws)
    kept = {k: v[-70:].cpu() for k, v in saved.items() if k != "kind"}
    z, u = H.decode(kept["gate"], kept["gate_scales"]), H.decode(kept["up"], kept["up_scales"])
    want = H.experts_backward(s.x[5:], *s.expert(2)[1], z, u, dy[-70:].cpu(), 0.0)
    H.check("dx", dx[-70:], *want["dx"])
