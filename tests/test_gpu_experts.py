"""The experts' products on sorted rows and their gradient on the GPU, against
float64 forms, expert by expert."""

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C
from tests import train_helpers as H

pytestmark = pytest.mark.gpu

GRADS = ("dx", "dw_gate", "dw_up", "dw_down")


def config(E, d, I, dtype, limit=0.0):
    return C.MoEConfig(dim=d, n_routed_experts=E, n_activated_experts=1, moe_inter_dim=I,
                       swiglu_limit=limit, act_dtype=dtype, expert_dtype=dtype)


class Step:
    """Inputs of a training step on the CPU, and its run on the GPU."""

    def __init__(self, counts, d, I, dtype, limit=0.0, spare=0, scale=1.0, seed=0):
        g, dt, E = H.gen(seed + 17 * d + I), H.TDT[dtype], len(counts)
        self.cfg, self.counts, self.dt = config(E, d, I, dtype, limit), counts, dt
        self.ends = [0]
        for n in counts:
            self.ends.append(self.ends[-1] + n)
        self.rows = self.ends[-1] + spare
        self.x = H.normal(g, dt, self.rows, d, std=scale)
        self.dy = H.normal(g, dt, self.rows, d)
        self.layer = {"w_gate": H.normal(g, dt, E, I, d, std=d ** -0.5),
                      "w_up": H.normal(g, dt, E, I, d, std=d ** -0.5),
                      "w_down": H.normal(g, dt, E, d, I, std=I ** -0.5)}

    def to(self, gpu, kind):
        self.kind = kind
        self.dev = {n: t.to(gpu) for n, t in self.layer.items()}
        self.x_d, self.dy_d = self.x.to(gpu), self.dy.to(gpu)
        self.off = torch.tensor(self.ends, dtype=torch.int32, device=gpu)
        self.ws = B.alloc_experts_workspace(self.cfg, self.rows, True, gpu)
        self.ws.fill_(0xFF)                                  # NaN, in both types
        self.saved = B.alloc_experts_saved(self.cfg, self.rows, kind, gpu)
        for t in self.saved.values():
            if isinstance(t, torch.Tensor):
                t.fill_(77)
        self.y = torch.full_like(self.x_d, -7.0)
        self.grads = {"dx": torch.full_like(self.x_d, -7.0),
                      **{"d" + n: torch.full_like(t, -7.0) for n, t in self.dev.items()}}
        return self

    def forward(self, **kw):
        B.moe_experts(self.cfg, self.dev, self.x_d, self.off, self.y, self.ws,
                      saved=None if self.kind == "none" else self.saved, **kw)

    def backward(self, names=GRADS, **kw):
        B.moe_experts_backward(self.cfg, self.dev, self.x_d, self.off, self.dy_d, self.saved,
                               {n: self.grads[n] for n in names}, self.ws, **kw)

    def expert(self, e):
        return slice(self.ends[e], self.ends[e + 1]), [self.layer[n][e] for n in
                                                       ("w_gate", "w_up", "w_down")]

    def kept(self, part):
        """The saved z and u of some rows, in float64."""
        s = {n: t.cpu() for n, t in self.saved.items() if isinstance(t, torch.Tensor)}
        if self.kind == "full":
            return s["gate"][part].double(), s["up"][part].double()
        return (H.decode(s["gate"][part], s["gate_scales"][part]),
                H.decode(s["up"][part], s["up_scales"][part]))

    def check_forward(self):
        limit = self.cfg.swiglu_limit
        y = self.y.cpu()
        for e, n in enumerate(self.counts):
            part, w = self.expert(e)
            if n == 0:
                continue
            f = H.experts_forward(self.x[part], *w, limit)
            H.check(f"y of expert {e}", y[part], *f["y"])
            if self.kind == "none":
                continue
            for name, got in zip(("z", "u"), self.kept(part)):
                want, tol = f[name]
                size = want.abs() + tol
                if self.kind == "full":
                    bound = tol + 2.0 ** -24 * size
                else:
                    # a step instead of half of one where rounding would cross the limit
                    steps = 2 if limit > 0 else 1
                    unit = torch.exp2(self.saved[{"z": "gate", "u": "up"}[name] + "_scales"]
                                      .cpu()[part].double() - 127).repeat_interleave(32, 1)
                    bound = tol + steps * torch.maximum(size * 2.0 ** -4, unit * 2.0 ** -10)
                H.check(f"saved {name} of expert {e}", got, want, bound)
                if limit > 0:
                    sure = (want.abs() - limit).abs() > tol
                    side = got > limit if name == "z" else got.abs() > limit
                    real = want > limit if name == "z" else want.abs() > limit
                    assert (side == real)[sure].all()
        assert (y[self.ends[-1]:] == -7).all()               # rows of no expert
        if self.kind != "none":
            for n in self.saved.values():
                if isinstance(n, torch.Tensor):
                    assert (n[self.ends[-1]:] == 77).all()

    def check_backward(self, names=GRADS):
        g = {n: t.cpu() for n, t in self.grads.items()}
        for e, n in enumerate(self.counts):
            part, w = self.expert(e)
            if n == 0:
                for name in names:
                    if name != "dx":
                        assert (g[name][e] == 0).all()
                continue
            want = H.experts_backward(self.x[part], *w, *self.kept(part), self.dy[part],
                                      self.cfg.swiglu_limit)
            for name in names:
                H.check(f"{name} of expert {e}", g[name][part] if name == "dx" else g[name][e],
                        *want[name])
        if "dx" in names:
            assert (g["dx"][self.ends[-1]:] == -7).all()


COUNTS = [
    ([1], 64, 32), ([0, 1, 0], 32, 64), ([5, 0, 3, 64, 65, 63], 72, 96), ([128, 1, 129, 127], 136, 32),
    ([200], 264, 160), ([0, 0, 300, 0], 64, 288), ([3] * 70, 16, 32), ([1, 0] * 100, 24, 32),
    ([257, 256, 255], 64, 128), ([40, 513, 7], 520, 224),
]


@pytest.mark.parametrize("dtype,kind", [("f32", "full"), ("f32", "mxfp8"), ("bf16", "full"),
                                        ("bf16", "mxfp8")])
@pytest.mark.parametrize("counts,d,I", COUNTS)
def test_training_step(gpu, counts, d, I, dtype, kind):
    print(f"[experts] rows={sum(counts)} E={len(counts)} d={d} I={I} {dtype} {kind}", flush=True)
    s = Step(counts, d, I, dtype, spare=9).to(gpu, kind)
    s.forward()
    s.check_forward()
    s.backward()
    s.check_backward()


@pytest.mark.parametrize("dtype,kind", [("f32", "full"), ("bf16", "full"), ("bf16", "mxfp8")])
@pytest.mark.parametrize("limit", [1.5, 10.0])
def test_clamp(gpu, limit, dtype, kind):
    s = Step([70, 0, 33], 96, 64, dtype, limit=limit, scale=limit / 2).to(gpu, kind)
    s.forward()
    s.check_forward()
    s.backward()
    s.check_backward()


@pytest.mark.parametrize("d,I", [(8, 8), (20, 36), (100, 52), (4, 4), (260, 12)])
def test_widths_of_whole_pieces(gpu, d, I):
    for dtype in ("f32", "bf16") if d % 8 == 0 and I % 8 == 0 else ("f32",):
        s = Step([17, 2, 90], d, I, dtype).to(gpu, "full")
        s.forward()
        s.check_forward()
        s.backward()
        s.check_backward()


def test_many_rows_of_one_expert(gpu):
    """46879 blocks of 64 rows: a block's number times the tiles' passes 31 bits."""
    s = Step([3_000_201, 7], 4, 4, "f32").to(gpu, "full")
    s.forward()
    s.backward()
    s.check_forward()
    s.check_backward()


def test_without_saving(gpu):
    s = Step([30, 2, 0, 70], 64, 96, "bf16", spare=4).to(gpu, "none")
    s.forward()
    s.check_forward()
    y = s.y.clone()
    s.to(gpu, "full").forward()
    assert torch.equal(s.y, y)                               # saving changes nothing


@pytest.mark.parametrize("names", [("dx",), ("dw_gate",), ("dw_up",), ("dw_down",),
                                   ("dw_gate", "dw_up"), ("dx", "dw_down")])
def test_gradients_alone(gpu, names):
    s = Step([30, 0, 70, 9], 64, 96, "bf16", spare=4).to(gpu, "mxfp8")
    s.forward()
    s.backward()
    s.check_backward()
    want = {n: s.grads[n].clone() for n in names}
    for t in s.grads.values():
        t.fill_(-7.0)
    s.ws.fill_(0xFF)
    s.backward(names)
    for n, t in s.grads.items():
        assert torch.equal(t, want[n]) if n in names else (t == -7).all(), n


def test_no_rows_at_all(gpu):
    s = Step([0, 0, 0], 64, 96, "bf16", spare=5).to(gpu, "mxfp8")
    s.forward()
    s.backward()
    s.check_forward()
    s.check_backward()
    empty = Step([0, 0], 64, 96, "f32").to(gpu, "full")
    empty.forward()
    empty.backward()
    assert all((empty.grads[n] == 0).all() for n in GRADS[1:])


def test_offsets_are_clamped(gpu):
    """Offsets outside the rows, or descending, reach no memory outside: what stands
    around the buffers stays."""
    s = Step([20, 30, 14], 64, 96, "bf16").to(gpu, "full")
    guard = torch.full((3, 64, 64), -7.0, dtype=torch.bfloat16, device=gpu)
    s.y = guard[1]
    for bad in ([0, 20, 50, 1000], [-5, 20, 50, 64], [0, 60, 30, 64], [2 ** 31 - 1, -2 ** 31, 7, 2 ** 31 - 1],
                [64, 64, 64, 64]):
        s.off = torch.tensor(bad, dtype=torch.int32, device=gpu)
        s.saved["gate"].fill_(0), s.saved["up"].fill_(0)
        s.forward()
        s.grads["dx"].fill_(0)
        s.backward()
        torch.cuda.synchronize()
        assert (guard[0] == -7).all() and (guard[2] == -7).all()


def test_not_finite_stays_with_its_rows(gpu):
    s = Step([10, 12], 64, 64, "bf16").to(gpu, "mxfp8")
    s.x_d[3, 5] = float("nan")
    s.forward()
    bad = ~torch.isfinite(s.y).all(1).cpu()
    assert bad[3] and bad.sum() == 1
    s.dy_d[15, 2] = float("inf")
    s.backward()
    bad = ~torch.isfinite(s.grads["dx"]).all(1).cpu()
    assert bad[3] and bad[15] and bad.sum() == 2


def whole(cfg, layer, x, T, gpu, state):
    """The routed experts' training step as a program runs it, on device tensors."""
    B.moe_route(cfg, layer, x, None, T, state["w"], state["idx"])
    B.moe_permute(cfg, state["idx"], T, state["counts"], state["off"], state["tok"], state["slot"],
                  state["inv"], None)
    B.moe_dispatch(cfg, x, state["inv"], T, state["xs"])
    B.moe_experts(cfg, layer, state["xs"], state["off"], state["ys"], state["ws"], saved=state["saved"])
    B.moe_combine(cfg, state["ys"], state["inv"], state["w"], T, state["y"], add=state["add"])
    B.moe_combine_backward(cfg, state["dy"], state["ys"], state["inv"], state["w"], T,
                           drows=state["dys"], dweights=state["dw"])
    B.moe_experts_backward(cfg, layer, state["xs"], state["off"], state["dys"], state["saved"],
                           state["grads"], state["ws"])
    B.moe_dispatch_backward(cfg, state["grads"]["dx"], state["inv"], T, state["dx"])


def whole_state(cfg, layer, T, gpu, kind, seed):
    d, k, E, dt = cfg.dim, cfg.n_activated_experts, cfg.n_routed_experts, H.TDT[cfg.act_dtype]
    i32 = dict(dtype=torch.int32, device=gpu)
    g = H.gen(seed)
    new = lambda *s: torch.zeros(s, dtype=dt, device=gpu)
    return {"w": torch.empty((T, k), device=gpu), "idx": torch.empty((T, k), **i32),
            "counts": torch.empty(E, **i32), "off": torch.empty(E + 1, **i32),
            "tok": torch.empty(T * k, **i32), "slot": torch.empty(T * k, **i32),
            "inv": torch.empty((T, k), **i32), "xs": new(T * k, d), "ys": new(T * k, d),
            "dys": new(T * k, d), "y": new(T, d), "dx": new(T, d),
            "dw": torch.empty((T, k), device=gpu), "ws": B.alloc_experts_workspace(cfg, T * k, True, gpu),
            "saved": B.alloc_experts_saved(cfg, T * k, kind, gpu),
            "add": H.normal(g, dt, T, d).to(gpu), "dy": H.normal(g, dt, T, d).to(gpu),
            "grads": {"dx": new(T * k, d), **{"d" + n: torch.empty_like(layer[n]) for n in
                                              ("w_gate", "w_up", "w_down")}}}


def layer_of(cfg, g, gpu):
    d, I, E, dt = cfg.dim, cfg.moe_inter_dim, cfg.n_routed_experts, H.TDT[cfg.act_dtype]
    return {"gate_w": H.normal(g, dt, E, d, std=d ** -0.5).to(gpu),
            "w_gate": H.normal(g, dt, E, I, d, std=d ** -0.5).to(gpu),
            "w_up": H.normal(g, dt, E, I, d, std=d ** -0.5).to(gpu),
            "w_down": H.normal(g, dt, E, d, I, std=I ** -0.5).to(gpu)}


def test_the_layer_together(gpu):
    """Route, permute, dispatch, experts, combine and their gradients in fp32, against
    torch's own gradient of the layer in float64, and against differences."""
    cfg = C.MoEConfig(dim=64, n_routed_experts=12, n_activated_experts=3, moe_inter_dim=96,
                      n_shared_experts=0, score_func="sigmoid", route_scale=1.5, swiglu_limit=2.0,
                      act_dtype="f32", expert_dtype="f32")
    g, T = H.gen(5), 150
    layer, x = layer_of(cfg, g, gpu), (torch.randn((T, 64), generator=g) * 2).to(gpu)
    s = whole_state(cfg, layer, T, gpu, "full", 6)
    whole(cfg, layer, x, T, gpu, s)

    idx, w = s["idx"].cpu().long(), s["w"].cpu().double().requires_grad_()
    leaves = {n: layer[n].cpu().double().requires_grad_() for n in ("w_gate", "w_up", "w_down")}
    xl = x.cpu().double().requires_grad_()

    def forward(xl, leaves, w):
        y = s["add"].cpu().double()
        for j in range(3):
            e = idx[:, j]
            z = torch.einsum("td,tid->ti", xl, leaves["w_gate"][e])
            u = torch.einsum("td,tid->ti", xl, leaves["w_up"][e])
            h = torch.nn.functional.silu(z.clamp(max=2.0)) * u.clamp(-2.0, 2.0)
            y = y + w[:, j:j + 1] * torch.einsum("ti,tdi->td", h, leaves["w_down"][e])
        return y

    y = forward(xl, leaves, w)
    dy = s["dy"].cpu().double()
    y.backward(dy)
    # fp32 sums of up to 96 and some 40 terms, each a product of three roundings:
    # 2^-24 times a hundred terms of the largest size met
    pairs = [("y", s["y"], y.detach()), ("dx", s["dx"], xl.grad), ("dw", s["dw"], w.grad)] + [
        (n, s["grads"]["d" + n], leaves[n].grad) for n in leaves]
    for name, got, want in pairs:
        H.check(name, got, want, 100 * 2.0 ** -24 * want.abs().max().expand_as(want))
    # differences of the device's own forward: in float64 sums of its fp32 outputs
    g2, step = H.gen(7), 2.0 ** -6
    for name, t, grad in (("w_down", layer["w_down"], s["grads"]["dw_down"]),
                          ("w_up", layer["w_up"], s["grads"]["dw_up"])):
        d = torch.randn(t.shape, generator=g2).to(gpu) * t.std() * 0.1
        grad = grad.clone().double()
        old, sums = t.clone(), []
        for sign in (1, -1):
            t.copy_(old + sign * step * d)
            B.moe_experts(cfg, layer, s["xs"], s["off"], s["ys"], s["ws"])
            B.moe_combine(cfg, s["ys"], s["inv"], s["w"], T, s["y"])
            sums.append((s["y"].double() * s["dy"].double()).sum().item())
        t.copy_(old)
        diff, want = (sums[0] - sums[1]) / (2 * step), (grad * d.double()).sum().item()
        # y is linear in either matrix but at the clamp, whose corner a value within
        # step * 0.1 of it can meet: those are below 1 % of the sum's size
        size = (grad.abs() * d.double().abs()).sum().item()
        assert abs(diff - want) < 1e-2 * size, (name, diff, want, size)


def test_forward_agrees_with_the_layer(gpu):
    """The same routed experts through moe_forward, in bf16: it rounds the weighted
    expert rows to bf16 and sums them in fp32, as these calls round rows and y."""
    cfg = C.MoEConfig(dim=128, n_routed_experts=16, n_activated_experts=4, moe_inter_dim=64,
                      n_shared_experts=0, score_func="sigmoid", swiglu_limit=10.0)
    g, T = H.gen(9), 333
    layer, x = layer_of(cfg, g, gpu), torch.randn((T, 128), generator=g).to(torch.bfloat16).to(gpu)
    s = whole_state(cfg, layer, T, gpu, "mxfp8", 4)
    s["add"].zero_()
    whole(cfg, layer, x, T, gpu, s)
    y = torch.empty_like(s["y"])
    ws = B.alloc_workspace(cfg, T, gpu)
    B.moe_forward(cfg, layer, x, None, T, y, ws)
    # each side: h within half a step twice over (2^-7 of the terms' norm at most),
    # rows and y half a step each
    err = (y.double() - s["y"].double()).abs().max().item()
    assert err <= 4 * 2.0 ** -8 * y.double().abs().max().item()


def test_captured_and_replayed(gpu):
    """A whole step in a HIP graph, replayed with other tokens (and so other
    offsets), with eager steps on the same weights between, on buffers of their own."""
    cfg = C.MoEConfig(dim=128, n_routed_experts=16, n_activated_experts=2, moe_inter_dim=64,
                      n_shared_experts=0, score_func="sigmoid", swiglu_limit=3.0)
    g, T = H.gen(11), 120
    layer = layer_of(cfg, g, gpu)
    xs = [torch.randn((T, 128), generator=g).to(torch.bfloat16).to(gpu) * (1 + i) for i in range(3)]
    x = xs[0].clone()
    s, eager = (whole_state(cfg, layer, T, gpu, "mxfp8", 3) for _ in range(2))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        whole(cfg, layer, x, T, gpu, s)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole(cfg, layer, x, T, gpu, s)
    for i in (1, 2, 0, 1, 1):
        whole(cfg, layer, xs[i], T, gpu, eager)
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((s, eager), (s["grads"], eager["grads"])):
            for n, t in a.items():
                if n in ("y", "dx", "dw", "dw_gate", "dw_up", "dw_down"):
                    assert torch.equal(t, b[n]), (i, n)


def test_two_streams_at_once(gpu):
    """Two steps on streams of their own, each with its workspace."""
    steps = [Step([90, 0, 300, 41], 128, 96, "bf16", seed=i).to(gpu, "mxfp8") for i in range(2)]
    for s in steps:
        s.forward()
        s.backward()
    torch.cuda.synchronize()
    want = [[s.y.clone()] + [t.clone() for t in s.grads.values()] for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s in steps:
            s.y.fill_(-7.0)
            for t in s.grads.values():
                t.fill_(-7.0)
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            s.forward(stream=stream)
            s.backward(stream=stream)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for a, b in zip([s.y] + list(s.grads.values()), w):
                assert torch.equal(a, b)
