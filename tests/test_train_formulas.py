"""The float64 forms that the GPU tests compare with, on the CPU: gradients against
differences, the 8-bit encoding against its definition."""

import pytest
import torch

from tests import train_helpers as H


@pytest.mark.parametrize("limit", [0.0, 0.7])
def test_experts_backward_against_differences(limit):
    g = H.gen(3)
    x, wg, wu, wd, dy = (torch.randn(s, generator=g, dtype=torch.float64).float() for s in (
        (5, 8), (6, 8), (6, 8), (8, 6), (5, 8)))

    def loss(x, wg, wu, wd):
        x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
        a, v, q, _, _ = H.halves(x @ wg.t(), x @ wu.t(), limit)
        return float(((a * q * v) @ wd.t() * dy.double()).sum())

    z, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    grads = H.experts_backward(x, wg, wu, wd, z, u, dy, limit)
    step = 2.0 ** -20                                        # kept by the fp32 inputs' doubles
    inputs = [t.double() for t in (x, wg, wu, wd)]
    for i, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        for _ in range(4):
            d = torch.randn(inputs[i].shape, generator=g, dtype=torch.float64)
            up, down = list(inputs), list(inputs)
            up[i], down[i] = inputs[i] + step * d, inputs[i] - step * d
            diff = (loss(*up) - loss(*down)) / (2 * step)
            want = float((grads[name][0] * d).sum())
            # second differences: step^2 times a third derivative of order 100; a
            # clamp's corner inside the step has not been met by these inputs
            assert abs(diff - want) < 1e-6 * (1 + abs(want)), name


def test_encode_is_the_nearest_value():
    g = H.gen(4)
    src = torch.randn((6, 70), generator=g) * torch.exp2(torch.randint(-20, 20, (6, 1), generator=g))
    codes, scales = H.encode(src)
    got = H.decode(codes, scales)
    unit = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :70]
    err = (got - src.double()).abs()
    assert (err <= torch.maximum(src.double().abs() * 2.0 ** -4, unit * 2.0 ** -10)).all()
    top = (src.double().abs() / unit).reshape(6, -1)
    assert (top <= 448).all()
    for b in range(3):                                       # and no smaller scale would hold
        assert (top[:, 32 * b:32 * b + 32].amax(1) > 224).all()


@pytest.mark.parametrize("limit", [10.0, 7.3, 0.001])
def test_encode_keeps_the_side_of_the_clamp(limit):
    g = H.gen(5)
    near = limit * (1 + torch.randn((64, 32), generator=g) * 0.05)
    near[:, 0] = limit
    got = H.decode(*H.encode(near, limit))
    assert ((got.abs() > limit) == (near.double().abs() > limit)).all()
    assert ((got - near.double()).abs() <= near.double().abs() / 7).all()   # a step at most


def test_permutation_is_one():
    inverse, R = H.permutation(20, 3, 8, H.gen(1), 0.2)
    rows = inverse[inverse >= 0].sort()[0]
    assert R < 60 and rows.tolist() == list(range(R))


@pytest.mark.parametrize("limit", [0.0, 7.0])
def test_encode_of_whole_blocks(limit):
    g = H.gen(6)
    src = torch.randn((40, 101), generator=g) * torch.exp2(torch.randint(-140, 100, (40, 1), generator=g))
    src[3] = 0.0
    src[::2] = torch.randn((20, 101), generator=g) * 7
    for dt in (torch.float32, torch.bfloat16):
        for a, b in zip(H.encode(src.to(dt), limit), H.encode_whole(src.to(dt), limit)):
            assert torch.equal(a, b)


def test_encode_at_the_top_of_the_range():
    top, step = 1.9375 * 2.0 ** 127, 2.0 ** 104               # fp32's step there
    src = torch.tensor([[top - step, -(top - step), 1.0, 0.0], [top, -top, 2.0 ** 127, 3.0],
                        [torch.finfo(torch.float32).max, 0.0, 0.0, 0.0]])
    codes, scales = H.encode(src)
    assert (scales == 247).all()
    back = H.decode(codes, scales).float()
    inf = src.abs() >= top
    assert (back.isinf() == inf).all() and (back[inf].sign() == src[inf].sign()).all()
    err = (back.double() - src.double()).abs()[~inf]
    assert (err <= torch.maximum(src.double().abs()[~inf] / 16, torch.tensor(2.0 ** 110))).all()
