"""moe_linear and moe_linear_backward against their float64 forms: every
activation and type, sizes from one row to several tiles with ragged and odd
widths, row strides, split contractions, empty batches, the clamp's border,
non-finite values, in-place residuals, graphs and streams, and a dense layer
followed by the MoE layer."""

import pytest
import torch

from mixture_experts_ffn_route_amd import binding as B
from mixture_experts_ffn_route_amd import config as C
from mixture_experts_ffn_route_amd import synth
from tests import linear_helpers as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]
# rows, in, out: single rows, one tile, ragged tiles, odd widths (padded rows),
# long contractions on few tiles (split), every tile shape
SIZES = [(1, 1, 1), (1, 16, 16), (1, 7, 5), (3, 8, 24), (16, 520, 264), (17, 33, 65), (64, 64, 64),
         (65, 97, 130), (200, 256, 320), (257, 300, 129), (300, 1000, 513), (64, 8192, 72),
         (90, 4099, 200), (1025, 96, 1032), (1500, 40, 700)]


def rand(shape, dt, gen, std=1.0, pad=0):
    wide = shape[:-1] + (shape[-1] + pad,)
    t = torch.empty(wide, dtype=torch.float32, device="cuda").normal_(0, std, generator=gen).to(dt)
    return t[..., :shape[-1]]


def make(M, K, N, dtype, activation, seed=0, bias=True, residual=True, limit=0.0, pad=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + M + 7 * K + 13 * N)
    dt = DT[dtype]
    two = activation == "swiglu"
    c = C.LinearConfig(M, K, N, dtype, activation, limit)
    t = dict(x=rand((M, K), dt, g, scale, pad), w=rand((N, K), dt, g, K ** -0.5).contiguous(),
             dy=rand((M, N), dt, g, 1.0, pad))
    if two:
        t["w_up"] = rand((N, K), dt, g, K ** -0.5).contiguous()
    if bias:
        t["bias"] = rand((N,), dt, g, 0.5)
        if two:
            t["bias_up"] = rand((N,), dt, g, 0.5)
    if residual:
        t["residual"] = rand((M, N), dt, g, 1.0, pad)
    return c, t


def workspace(c, t, backward=False):
    ld = {"ld_x": t["x"].stride(0), "ld_y": t["dy"].stride(0)}
    if "residual" in t:
        ld["ld_residual"] = t["residual"].stride(0)
    ws = B.alloc_linear_workspace(c, backward, **ld)
    return ws.fill_(0xFF)                          # NaN patterns: nothing may be read unwritten


def outputs(c, t, pad=0, keep=True):
    dt = DT[c.dtype]
    y = torch.full((c.rows, c.out_dim + pad), float("nan"), dtype=dt, device="cuda")[:, :c.out_dim]
    z = torch.full((c.rows, c.out_dim), float("nan"), dtype=dt, device="cuda") if keep else None
    zu = torch.full_like(z, float("nan")) if keep and c.activation == "swiglu" else None
    return y, z, zu


def run(c, t, y, z, zu, ws, stream=None):
    opt = {n: t.get(n) for n in ("bias", "residual", "w_up", "bias_up")}
    B.moe_linear(c, t["x"], t["w"], y, z=z, z_up=zu, ws=ws, stream=stream, **opt)


def run_backward(c, t, z, zu, ws, names, stream=None, dy=None):
    M, K, N, dt = c.rows, c.in_dim, c.out_dim, DT[c.dtype]
    shape = {"dx": (M, K), "dw": (N, K), "dw_up": (N, K), "dbias": (N,), "dbias_up": (N,)}
    out = {n: torch.full(shape[n], float("nan"), dtype=dt, device="cuda") for n in names}
    if "dx" in out:                                # rows at x's stride
        wide = torch.full((M, max(t["x"].stride(0), K)), float("nan"), dtype=dt, device="cuda")
        out["dx"] = wide[:, :K]
    B.moe_linear_backward(c, t["dy"] if dy is None else dy, t["x"], t["w"], w_up=t.get("w_up"), z=z,
                          z_up=zu, ws=ws, stream=stream, **out)
    return out


def grad_names(c):
    two = c.activation == "swiglu"
    return ["dx", "dw", "dbias"] + (["dw_up", "dbias_up"] if two else [])


def check_all(c, t, label, pad=0):
    y, z, zu = outputs(c, t, t["dy"].stride(0) - c.out_dim if c.rows > 1 else 0)
    ws = workspace(c, t, True)
    print(f"[linear] {label}", flush=True)
    run(c, t, y, z, zu, ws)
    torch.cuda.synchronize()
    opt = {n: t.get(n) for n in ("bias", "residual", "w_up", "bias_up")}
    ref, tol, rz, ez, ru, eu = R.forward(c, t["x"], t["w"], **opt)
    R.check(f"{label} y", y, ref, tol)
    half = R.HALF[DT[c.dtype]]
    R.check(f"{label} z", z, rz, ez + 2 * half * rz.abs() + 1e-30)   # one step at the clamp's border
    if zu is not None:
        R.check(f"{label} z_up", zu, ru, eu + 2 * half * ru.abs() + 1e-30)
    ws.fill_(0xFF)
    names = grad_names(c)
    got = run_backward(c, t, z, zu, ws, names)
    torch.cuda.synchronize()
    want = R.backward(c, t["dy"], t["x"], t["w"], z, t.get("w_up"), zu)
    for n in names:
        R.check(f"{label} {n}", got[n], *want[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("activation", ["silu", "swiglu"])
def test_sizes(M, K, N, activation, dtype, gpu):
    c, t = make(M, K, N, dtype, activation)
    check_all(c, t, f"{dtype} {activation} {M}x{K}x{N}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (False, False)])
def test_activations(activation, bias, residual, dtype, gpu):
    c, t = make(77, 200, 104, dtype, activation, 3, bias, residual, scale=3.0)
    check_all(c, t, f"{dtype} {activation} bias={bias} residual={residual}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,pad", [(33, 64, 48, 8), (130, 64, 48, 5), (5, 40, 72, 1), (9, 31, 17, 4)])
@pytest.mark.parametrize("activation", ["none", "swiglu", "gelu"])
def test_row_strides(M, K, N, pad, activation, dtype, gpu):
    c, t = make(M, K, N, dtype, activation, 5, pad=pad)
    check_all(c, t, f"{dtype} {activation} {M}x{K}x{N} pad {pad}")


@pytest.mark.parametrize("dtype,M,K,N", [("bf16", 4096, 192, 4096), ("bf16", 4100, 328, 1500),
                                         ("f32", 2300, 130, 2050), ("bf16", 8200, 64, 520)])
@pytest.mark.parametrize("activation", ["none", "swiglu"])
def test_large(dtype, M, K, N, activation, gpu):
    c, t = make(M, K, N, dtype, activation, 6)
    check_all(c, t, f"{dtype} {activation} {M}x{K}x{N}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("limit", [1.0, 0.7, 10.0])
def test_clamp(dtype, limit, gpu):
    c, t = make(150, 96, 80, dtype, "swiglu", 7, limit=limit, scale=4.0)
    check_all(c, t, f"{dtype} clamp {limit}")


@pytest.mark.parametrize("limit", [1.0, 0.7, 3.3])
def test_saved_values_keep_the_side_of_the_clamp(limit, gpu):
    """Pre-activations a fraction of a bf16 step around the border: the saved
    bf16 value is on the side the fp32 one was (K = 2 sums that are exact)."""
    steps = torch.arange(-40, 41, device="cuda").float() * 2.0 ** -10
    top = torch.tensor([limit, -limit], device="cuda").repeat_interleave(steps.numel())
    want = top + torch.cat([steps, steps]) * limit
    hi = want.to(torch.bfloat16)
    lo = (want - hi.float()).to(torch.bfloat16)
    exact = hi.double() + lo.double()
    M = want.numel()
    x = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = hi, lo
    w = torch.zeros((8, 8), dtype=torch.bfloat16, device="cuda")
    w[:, 0] = w[:, 1] = 1
    c = C.LinearConfig(M, 8, 8, "bf16", "swiglu", limit)
    y, z, zu = outputs(c, {})
    B.moe_linear(c, x, w, y, w_up=w, z=z, z_up=zu, ws=B.alloc_linear_workspace(c))
    torch.cuda.synchronize()
    L = float(torch.tensor(limit, dtype=torch.float32))
    assert torch.equal(z[:, 0].double() > L, exact > L)
    assert torch.equal(zu[:, 0].double().abs() > L, exact.abs() > L)
    assert ((z[:, 0].double() - exact).abs() <= 2.0 ** -7 * exact.abs()).all()


@pytest.mark.parametrize("activation", ["none", "swiglu"])
def test_no_rows(activation, gpu):
    c, t = make(0, 24, 40, "bf16", activation)
    ws = workspace(c, {"x": t["x"], "dy": t["dy"]}, True)
    y, z, zu = outputs(c, t)
    run(c, t, y, z, zu, ws)
    got = run_backward(c, t, z, zu, ws, grad_names(c))
    torch.cuda.synchronize()
    for n in grad_names(c):
        assert not got[n].any(), n                 # zeros, not what was there
    assert got["dx"].numel() == 0


def test_residual_in_place(gpu):
    for M, K, N in ((5, 64, 72), (300, 128, 264), (70, 4096, 96)):
        c, t = make(M, K, N, "bf16", "none", 9)
        y, _, _ = outputs(c, t, keep=False)
        ws = workspace(c, t)
        run(c, t, y, None, None, ws)
        stream = t["residual"].contiguous().clone()
        run(c, dict(t, residual=stream), stream, None, None, ws)
        torch.cuda.synchronize()
        assert torch.equal(stream, y)


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_row_stays_in_its_row(M, value, gpu):
    c, t = make(M, 72, 88, "bf16", "silu", 11)
    ws = workspace(c, t, True)
    y0, z0, _ = outputs(c, t)
    run(c, t, y0, z0, None, ws)
    x = t["x"].clone()
    x[2, 5] = value
    y1, z1, _ = outputs(c, t)
    run(c, dict(t, x=x), y1, z1, None, ws)
    torch.cuda.synchronize()
    keep = [i for i in range(M) if i != 2]
    assert torch.equal(y1[keep], y0[keep])
    assert not torch.isfinite(y1[2].float()).all()


def test_rows_and_columns_outside_are_left_alone(gpu):
    """Buffers wider and longer than the call: the frame keeps its values."""
    M, K, N = 70, 48, 56
    c, t = make(M, K, N, "bf16", "swiglu", 12)
    frame = torch.full((M + 4, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    y = frame[2:M + 2, 8:N + 8]
    _, z, zu = outputs(c, t)
    ld = dict(ld_y=N + 16)
    run(c, t, y, z, zu, B.alloc_linear_workspace(c, **ld))
    torch.cuda.synchronize()
    inner = torch.zeros_like(frame, dtype=torch.bool)
    inner[2:M + 2, 8:N + 8] = True
    assert (frame[~inner] == 7.0).all()
    ref, tol, *_ = R.forward(c, t["x"], t["w"], t["bias"], t["residual"], t["w_up"], t["bias_up"])
    R.check("framed y", y, ref, tol)


def test_gradients_one_at_a_time(gpu):
    """Each gradient alone equals the one of the full call."""
    for act in ("none", "swiglu"):
        c, t = make(150, 72, 96, "bf16", act, 13)
        ws = workspace(c, t, True)
        y, z, zu = outputs(c, t)
        run(c, t, y, z, zu, ws)
        full = run_backward(c, t, z, zu, ws, grad_names(c))
        for n in grad_names(c):
            ws.fill_(0xFF)
            one = run_backward(c, t, z, zu, ws, [n])
            torch.cuda.synchronize()
            assert torch.equal(one[n], full[n]), (act, n)


@pytest.mark.parametrize("activation", ACTS)
def test_gradient_against_differences(activation, gpu):
    """fp32 gradients along random directions against central differences of
    the float64 forward (step h: error h^2 of the third derivative)."""
    c, t = make(20, 24, 16, "f32", activation, 15, limit=2.0 if activation == "swiglu" else 0.0)
    ws = workspace(c, t, True)
    y, z, zu = outputs(c, t)
    run(c, t, y, z, zu, ws)
    got = run_backward(c, t, z, zu, ws, grad_names(c))
    torch.cuda.synchronize()
    wide = {n: v.double() for n, v in t.items() if n != "dy"}

    def loss(p):
        zz = p["x"].mm(p["w"].t()) + p["bias"]
        if activation == "swiglu":
            g, v, _, _ = R.clamped(zz, p["x"].mm(p["w_up"].t()) + p["bias_up"], c.limit)
            out = g / (1 + torch.exp(-g)) * v
        else:
            out = R.act(zz, activation)
        return ((out + p["residual"]) * t["dy"].double()).sum().item()

    h = 1e-6
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for n in grad_names(c):
        v = torch.empty_like(wide[n[1:]]).normal_(generator=g)
        d = (loss({**wide, n[1:]: wide[n[1:]] + h * v}) -
             loss({**wide, n[1:]: wide[n[1:]] - h * v})) / (2 * h)
        got_d = (got[n].double() * v).sum().item()
        scale = (got[n].double() * v).abs().sum().item()
        # a kink (relu, clamp) within h of a value moves one term by h; fp64
        # differences are good to 1e-9 / h of the loss
        assert abs(d - got_d) <= 2e-5 * scale + 1e-3, (n, d, got_d)


def test_graph_replays_of_a_training_step(gpu):
    c, t = make(140, 96, 80, "bf16", "swiglu", 17)
    ws = workspace(c, t, True)
    y, z, zu = outputs(c, t)
    xs = [t["x"].clone(), (t["x"] * -0.5).contiguous()]
    x = t["x"].clone()
    ts = dict(t, x=x)
    grads = {n: torch.empty_like(v) for n, v in
             run_backward(c, ts, *_saved(c, ts, ws), ws, grad_names(c)).items()}

    def step():
        run(c, ts, y, z, zu, ws)
        B.moe_linear_backward(c, t["dy"], x, t["w"], w_up=t["w_up"], z=z, z_up=zu, ws=ws, **grads)

    refs = []
    for src in xs:
        x.copy_(src)
        step()
        torch.cuda.synchronize()
        refs.append([v.clone() for v in (y, *grads.values())])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(4):
        x.copy_(xs[r % 2])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, *grads.values()), refs[r % 2]):
            assert torch.equal(a, b), r
        run(c, t, *outputs(c, t), workspace(c, t))     # eager work between the replays
        torch.cuda.synchronize()


def _saved(c, t, ws):
    y, z, zu = outputs(c, t)
    run(c, t, y, z, zu, ws)
    return z, zu


def test_two_streams(gpu):
    c, t = make(200, 4096, 96, "bf16", "gelu", 19)
    ref, _, _ = outputs(c, t, keep=False)
    run(c, t, ref, None, None, workspace(c, t))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [workspace(c, t) for _ in range(2)]
    outs = [[outputs(c, t, keep=False)[0] for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(6):
        for i in range(2):
            run(c, t, outs[i][j], None, None, wss[i], streams[i])
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, ref)


def test_dense_layer_then_moe_layer(gpu):
    """A decode step of a dense SwiGLU layer on the residual stream, then the
    MoE layer for the same tokens; the dense layer's training step."""
    wl = C.SMALL_WORKLOADS["v3_small"]
    cfg, T, d, I = wl.cfg, 6, wl.cfg.dim, 320
    layer = synth.make_layer(wl, gpu)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = layer["x"][:T].contiguous()
    wg, wu = (rand((I, d), torch.bfloat16, g, d ** -0.5).contiguous() for _ in range(2))
    wd = rand((d, I), torch.bfloat16, g, I ** -0.5).contiguous()
    up = C.LinearConfig(T, d, I, "bf16", "swiglu", 10.0)
    down = C.LinearConfig(T, I, d, "bf16")
    h, zg, zu = (torch.empty((T, I), dtype=torch.bfloat16, device=gpu) for _ in range(3))
    y = torch.empty_like(x)
    ws = B.alloc_linear_workspace(up, True)
    ws2 = B.alloc_linear_workspace(down, True)
    B.moe_linear(up, x, wg, h, w_up=wu, z=zg, z_up=zu, ws=ws)
    B.moe_linear(down, h, wd, y, residual=x, ws=ws2)
    out = torch.empty_like(x)
    B.moe_forward_few(cfg, layer, y, None, T, out, B.alloc_few_workspace(cfg, T, gpu))
    ref_out = torch.empty_like(x)
    B.moe_forward(cfg, layer, y, None, T, ref_out, B.alloc_workspace(cfg, T, gpu))
    dy = torch.ones_like(y)
    dh, dwd = torch.empty_like(h), torch.empty_like(wd)
    B.moe_linear_backward(down, dy, h, wd, dx=dh, dw=dwd, ws=ws2)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    B.moe_linear_backward(up, dh, x, wg, w_up=wu, z=zg, z_up=zu, dx=dx, dw=dwg, dw_up=dwu, ws=ws)
    torch.cuda.synchronize()
    rh, th, *_ = R.forward(up, x, wg, w_up=wu)
    R.check("dense h", h, rh, th)
    ry, ty, *_ = R.forward(down, h, wd, residual=x)
    R.check("dense y", y, ry, ty)
    assert float((out.float() - ref_out.float()).abs().max()) <= 2e-2 * float(ref_out.float().abs().max())
    want = R.backward(down, dy, h, wd)
    R.check("dh", dh, *want["dx"])
    R.check("dwd", dwd, *want["dw"])
    want = R.backward(up, dh, x, wg, zg, wu, zu)
    for n, v in (("dx", dx), ("dw", dwg), ("dw_up", dwu)):
        R.check(n, v, *want[n])
