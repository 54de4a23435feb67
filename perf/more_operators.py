"""What is timed of the operators that train the MoE layer: token rows to their
experts and back with the gate values, 8-bit checkpoints of activations, and the
experts' products on sorted rows, each with its gradient.

``own`` chooses between the plain torch form of each (32-bit arithmetic on the
same inputs) and the HIP kernels as a program calls them.
"""

import math

import torch

own = False

DEV = "cuda"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _sort(name, op, tokens, dim, slots, experts, dtype="bf16", add=False, dropped=0.0):
    return dict(op=op, tokens=tokens, dim=dim, slots=slots, experts=experts, dtype=dtype, add=add,
                dropped=dropped, name=name)


def _keep(name, rows, cols, dtype="bf16", limit=0.0, pad=0):
    return dict(op="keep", rows=rows, cols=cols, dtype=dtype, limit=limit, pad=pad, name=name)


def _experts(name, op, rows, experts, dim, inter, dtype="bf16", save="none", limit=0.0, scale=1.0,
             spare=0):
    return dict(op=op, rows=rows, experts=experts, dim=dim, inter=inter, dtype=dtype, save=save,
                limit=limit, scale=scale, spare=spare, name=name)


def listed():
    return [
        # a decode batch's rows on their way to the experts' ranks: latency
        _sort("dispatch_decode", "dispatch", 64, 7168, 8, 256),
        # gradient of the rows of a training batch, summed back to its tokens
        _sort("dispatch_grad_flash", "dispatch_grad", 8192, 5120, 8, 384),
        # an fp32 model with an odd width and a capacity that drops some pairs
        _sort("combine_odd_f32", "combine", 203, 1001, 3, 16, dtype="f32", dropped=0.1),
        # the experts' rows of a prompt weighted, summed and added to the shared expert's
        _sort("combine_v3", "combine", 4096, 7168, 8, 256, add=True),
        # gradients of rows and gate values of a training batch
        _sort("combine_grad_hash", "combine_grad", 4096, 2048, 4, 64, dropped=0.02),
        # pre-activations of a small layer, in rows of a wider buffer, kept and read back
        _keep("keep_odd_f32", 77, 777, dtype="f32", limit=10.0, pad=5),
        # pre-activations of a training batch with the clamp
        _keep("keep_flash", 65536, 1536, limit=10.0),
        # a test-sized fp32 layer: nothing but latency
        _experts("experts_tiny_f32", "experts", 128, 16, 128, 64, dtype="f32"),
        # a decode batch on one of eight ranks: a stream of that rank's weights
        _experts("experts_decode_v3", "experts", 64, 32, 7168, 2048),
        # a small fp32 training step, pre-activations kept as they are
        _experts("train_small_f32", "train", 1003, 8, 256, 192, dtype="f32", save="full", spare=21),
        # a training step at the hash workload's widths and rows
        _experts("train_hash_width", "train", 16384, 64, 2048, 1024, save="mxfp8"),
        # one rank's share of eight of the V4.1-Flash workload, the clamp active: the largest
        _experts("train_flash_share", "train", 8192, 48, 5120, 1536, save="mxfp8", limit=10.0,
                 scale=4.0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.4:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        dim = _logint(rng, 16, 2048 if dtype == "f32" else 7168)
        if rng.random() < 0.7:
            dim = max(64, dim // 64 * 64)
        slots = rng.randint(1, 8)
        return dict(op=rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad"]),
                    tokens=_logint(rng, 1, 8192), dim=dim, slots=slots,
                    experts=rng.choice([8, 16, 64, 256]), dtype=dtype, add=rng.random() < 0.5,
                    dropped=rng.choice([0.0, 0.0, 0.05]))
    if kind < 0.55:
        return dict(op="keep", rows=_logint(rng, 1, 65536), cols=_logint(rng, 8, 2048),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), limit=rng.choice([0.0, 10.0, 7.0]),
                    pad=rng.choice([0, 0, 8, 3]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    small = dtype == "f32"
    op = rng.choice(["experts", "train", "train"])
    # fp32 layers keep all bits: 8 bits of values next to a border would show
    save = "none" if op == "experts" else "full" if small else rng.choice(["full", "mxfp8"])
    unit = 32 if save == "mxfp8" else 4 if small else 8
    dim = max(16, _logint(rng, 64, 1024 if small else 7168) // 8 * 8)
    inter = max(unit, _logint(rng, 32, 1024 if small else 2048) // unit * unit)
    experts = rng.choice([4, 8, 16, 33, 64])
    experts = max(1, min(experts, 48 * 5120 * 1536 // (dim * inter)))
    rows = min(_logint(rng, 1, 2048 if small else 16384), 8192 * 5120 * 1536 // (dim * inter))
    limit = rng.choice([0.0, 10.0])
    return dict(op=op, rows=rows, experts=experts, dim=dim, inter=inter, dtype=dtype, save=save,
                limit=limit, scale=rng.choice([1.0, 4.0]), spare=rng.choice([0, 0, 17]))


# ---- inputs ----------------------------------------------------------------

def _gen(seed, tag, device=None):
    g = torch.Generator(device=device or DEV)
    g.manual_seed((int(seed) * 1000003 + tag * 7919 + 29) % (1 << 62))
    return g


def _normal(shape, dtype, std, g):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _permutation(c, seed):
    """Row of each (token, slot) pair sorted by expert, -1: dropped, and the
    number of rows: what a routing of the batch gives."""
    T, E, k = c["tokens"], c["experts"], c["slots"]
    like = 0.5 * torch.randn(E, device=DEV, generator=_gen(seed, 1))
    noise = torch.rand((T, E), device=DEV, generator=_gen(seed, 2))
    expert = (like - torch.log(-torch.log(noise))).topk(k, dim=1)[1].reshape(-1)
    if c["dropped"]:
        out = torch.rand(T * k, device=DEV, generator=_gen(seed, 3)) < c["dropped"]
        expert = torch.where(out, E, expert)
    order = expert.sort(stable=True)[1]
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(T * k, device=DEV)
    inverse = torch.where(expert < E, inverse, -1).to(torch.int32).reshape(T, k)
    return inverse.contiguous()


def _prepare_sort(c, seed):
    T, d, k, dt = c["tokens"], c["dim"], c["slots"], TDT[c["dtype"]]
    s = {"case": c, "inverse": _permutation(c, seed)}
    op = c["op"]
    if op in ("dispatch", "combine_grad"):
        s["x"] = _normal((T, d), dt, 1.0, _gen(seed, 4))         # x, or the gradient of y
    if op != "dispatch":
        s["rows"] = _normal((T * k, d), dt, 1.0, _gen(seed, 5))  # the experts' rows, or their gradient
    if op in ("combine", "combine_grad"):
        w = torch.rand((T, k), device=DEV, generator=_gen(seed, 6)) + 0.1
        s["weights"] = w / w.sum(dim=1, keepdim=True)
    if op == "combine" and c["add"]:
        s["add"] = _normal((T, d), dt, 1.0, _gen(seed, 7))
    if own:
        from mixture_experts_ffn_route_amd import binding, config
        s["B"] = binding
        s["cfg"] = binding.config_c(config.MoEConfig(
            dim=d, n_routed_experts=c["experts"], n_activated_experts=k, moe_inter_dim=64,
            act_dtype=c["dtype"], expert_dtype=c["dtype"]))
        if op in ("dispatch", "combine_grad"):
            s["out"] = torch.zeros((T * k, d), dtype=dt, device=DEV)
        else:
            s["out"] = torch.empty((T, d), dtype=dt, device=DEV)
        if op == "combine_grad":
            s["dweights"] = torch.empty((T, k), device=DEV)
    return s


def _prepare_keep(c, seed):
    rows, cols, dt = c["rows"], c["cols"], TDT[c["dtype"]]
    # some columns are larger than others, as features of a layer are
    std = torch.exp(torch.randn(cols + c["pad"], device=DEV, generator=_gen(seed, 1)))
    src = (_normal((rows, cols + c["pad"]), torch.float32, 1.0, _gen(seed, 2)).mul_(std * 2.0)).to(dt)
    s = {"case": c, "src": src[:, :cols]}
    if own:
        from mixture_experts_ffn_route_amd import binding
        s["B"] = binding
        s["codes"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((rows, -(-cols // 32)), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((rows, cols), dtype=dt, device=DEV)
    return s


def _prepare_experts(c, seed):
    R, E, d, I, dt = c["rows"], c["experts"], c["dim"], c["inter"], TDT[c["dtype"]]
    g = _gen(seed, 1, "cpu")
    like = torch.softmax(0.5 * torch.randn(E, generator=g), dim=0)
    counts = torch.bincount(torch.multinomial(like, R, replacement=True, generator=g), minlength=E)
    ends = [0] + counts.cumsum(0).tolist()
    L = {"w_gate": _normal((E, I, d), dt, d ** -0.5, _gen(seed, 2)),
         "w_up": _normal((E, I, d), dt, d ** -0.5, _gen(seed, 3)),
         "w_down": _normal((E, d, I), dt, I ** -0.5, _gen(seed, 4))}
    # rows past the last expert's are room that this batch does not use
    s = {"case": c, "layer": L, "ends": ends,
         "x": _normal((R + c["spare"], d), dt, c["scale"], _gen(seed, 5))}
    train = c["op"] == "train"
    if train:
        s["dy"] = _normal((R + c["spare"], d), dt, 1.0, _gen(seed, 6))
    if own:
        from mixture_experts_ffn_route_amd import binding, config
        cfg = config.MoEConfig(dim=d, n_routed_experts=E, n_activated_experts=1, moe_inter_dim=I,
                               swiglu_limit=c["limit"], act_dtype=c["dtype"],
                               expert_dtype=c["dtype"])
        s["B"], s["cfg"], s["weights"] = binding, binding.config_c(cfg), binding.weights_c(L)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        s["ws"] = binding.alloc_experts_workspace(cfg, R + c["spare"], backward=train)
        s["y"] = torch.zeros((R + c["spare"], d), dtype=dt, device=DEV)
        s["saved"] = binding.alloc_experts_saved(cfg, R + c["spare"], c["save"]) if train else None
        if train:
            s["grads"] = {"dx": torch.zeros_like(s["x"]), **{"d" + n: torch.empty_like(L[n]) for n in L}}
    return s


def prepare(case, seed):
    if case["op"] == "keep":
        return _prepare_keep(case, seed)
    return (_prepare_experts if case["op"] in ("experts", "train") else _prepare_sort)(case, seed)


# ---- the plain forms -------------------------------------------------------

def _plain_sort(s):
    c, inverse = s["case"], s["inverse"].long()
    T, k = inverse.shape
    dt, d = TDT[c["dtype"]], c["dim"]
    there, at = inverse >= 0, inverse.clamp(min=0)
    if c["op"] == "dispatch":
        out = torch.zeros((T * k, d), dtype=dt, device=DEV)
        out[inverse[there]] = s["x"].repeat_interleave(k, dim=0)[there.reshape(-1)]
        return {"rows": out}
    if c["op"] in ("dispatch_grad", "combine"):
        y = torch.zeros((T, d), device=DEV)
        for j in range(k):
            w = there[:, j].float()
            if c["op"] == "combine":
                w = w * s["weights"][:, j]
            y += w.unsqueeze(1) * s["rows"][at[:, j]].float()
        if c["op"] == "combine" and c["add"]:
            y += s["add"].float()
        return {"y": y.to(dt)}
    drows = torch.zeros((T * k, d), dtype=dt, device=DEV)
    dweights = torch.zeros((T, k), device=DEV)
    dy = s["x"].float()
    for j in range(k):
        m = there[:, j]
        drows[inverse[m, j]] = (s["weights"][m, j].unsqueeze(1) * dy[m]).to(dt)
        dweights[:, j] = (s["rows"][at[:, j]].float() * dy).sum(dim=1) * m
    return {"drows": drows, "dweights": dweights}


def _kept(v, limit):
    """fp32 rows as the 8-bit values that are kept of them: E4M3 times a power of
    two a block of 32 columns, the least one that holds the block's largest
    value; nothing is rounded across the limit."""
    rows, cols = v.shape
    full = torch.zeros((rows, -(-cols // 32) * 32), device=v.device)
    full[:, :cols] = v
    b = full.reshape(rows, -1, 32)
    top = b.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(top)
    x = torch.where(top > 0, e - 9 + (m > 0.875), 0).clamp(-127, 127)
    unit = torch.exp2(x.float())
    q = (b / unit).to(torch.float8_e4m3fn)
    if limit > 0:
        over, is_over = b.abs() > limit, (q.float() * unit).abs() > limit
        q = (q.view(torch.uint8) + (over & ~is_over).to(torch.uint8) -
             (is_over & ~over).to(torch.uint8)).view(torch.float8_e4m3fn)
    return (q.float() * unit).reshape(rows, -1)[:, :cols]


def _plain_experts(s):
    c, L, ends = s["case"], s["layer"], s["ends"]
    train, dt = c["op"] == "train", s["x"].dtype
    top = c["limit"] if c["limit"] > 0 else math.inf
    out = {"y": torch.zeros_like(s["x"])}
    if train:
        out["dx"] = torch.zeros_like(s["x"])
        out.update({"d" + n: torch.zeros_like(L[n]) for n in L})
    for e in range(c["experts"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        x = s["x"][lo:hi].float()
        gate, up, down = (L[n][e].float() for n in ("w_gate", "w_up", "w_down"))
        z, u = x @ gate.t(), x @ up.t()
        g, v = z.clamp(max=top), u.clamp(-top, top)
        out["y"][lo:hi] = ((g * torch.sigmoid(g) * v) @ down.t()).to(dt)
        if not train:
            continue
        if c["save"] == "mxfp8":
            z, u = _kept(z, c["limit"]), _kept(u, c["limit"])
        g, v = z.clamp(max=top), u.clamp(-top, top)
        p = torch.sigmoid(g)
        dy = s["dy"][lo:hi].float()
        dh = dy @ down
        dz = dh * v * p * (1 + g * (1 - p)) * (z <= top)
        du = dh * g * p * (u.abs() <= top)
        out["dx"][lo:hi] = (dz @ gate + du @ up).to(dt)
        out["dw_gate"][e] = (dz.t() @ x).to(dt)
        out["dw_up"][e] = (du.t() @ x).to(dt)
        out["dw_down"][e] = (dy.t() @ (g * p * v)).to(dt)
    return out


# ---- one pass --------------------------------------------------------------

def _own_sort(s):
    B, c, T = s["B"], s["case"], s["case"]["tokens"]
    if c["op"] == "dispatch":
        B.moe_dispatch(s["cfg"], s["x"], s["inverse"], T, s["out"])
        return {"rows": s["out"]}
    if c["op"] == "dispatch_grad":
        B.moe_dispatch_backward(s["cfg"], s["rows"], s["inverse"], T, s["out"])
        return {"y": s["out"]}
    if c["op"] == "combine":
        B.moe_combine(s["cfg"], s["rows"], s["inverse"], s["weights"], T, s["out"], add=s.get("add"))
        return {"y": s["out"]}
    B.moe_combine_backward(s["cfg"], s["x"], s["rows"], s["inverse"], s["weights"], T,
                           drows=s["out"], dweights=s["dweights"])
    return {"drows": s["out"], "dweights": s["dweights"]}


def _own_keep(s):
    s["B"].moe_checkpoint_save(s["src"], s["codes"], s["scales"], limit=s["case"]["limit"])
    s["B"].moe_checkpoint_load(s["codes"], s["scales"], s["out"])
    return {"values": s["out"]}


def _own_experts(s):
    B = s["B"]
    B.moe_experts(s["cfg"], s["weights"], s["x"], s["offsets"], s["y"], s["ws"], saved=s["saved"])
    if s["case"]["op"] == "experts":
        return {"y": s["y"]}
    B.moe_experts_backward(s["cfg"], s["weights"], s["x"], s["offsets"], s["dy"], s["saved"],
                           s["grads"], s["ws"])
    return {"y": s["y"], **s["grads"]}


def run(state):
    op = state["case"]["op"]
    if op == "keep":
        if own:
            return _own_keep(state)
        v = state["src"]
        return {"values": _kept(v.float(), state["case"]["limit"]).to(v.dtype)}
    if op in ("experts", "train"):
        return (_own_experts if own else _plain_experts)(state)
    return (_own_sort if own else _plain_sort)(state)


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "keep":
        # written and read back: values in, codes and scales out and in, values out
        n = c["rows"] * c["cols"]
        return {"bytes": int(n * (2 * size + 2 * (1 + 1 / 32))), "flops": 4 * n}
    if c["op"] in ("experts", "train"):
        R, E, d, I = c["rows"], c["experts"], c["dim"], c["inter"]
        weights = 3 * d * I
        hit = E * (1.0 - (1.0 - 1.0 / E) ** R)                   # experts with rows, expected
        if c["op"] == "experts":
            return {"bytes": int((2 * R * d + hit * weights) * size), "flops": 2 * weights * R}
        # x, dy and the weights read, y, dx and every expert's gradients written
        return {"bytes": int((4 * R * d + (hit + E) * weights) * size), "flops": 6 * weights * R}
    T, d, k = c["tokens"], c["dim"], c["slots"]
    pairs = int(T * k * (1.0 - c["dropped"]))
    index = 4 * T * k
    tokens = T * d * (2 if c["op"] == "combine" and c["add"] else 1)
    if c["op"] == "combine_grad":
        return {"bytes": (tokens + 2 * pairs * d) * size + 3 * index, "flops": 3 * pairs * d}
    return {"bytes": (tokens + pairs * d) * size + index * (2 if c["op"] == "combine" else 1),
            "flops": 2 * pairs * d}


# ---- the definition in 64 bits ---------------------------------------------

def _exact_sort(c, s):
    inverse = s["inverse"].long().reshape(-1)
    T, k, d = c["tokens"], c["slots"], c["dim"]
    pair = (inverse >= 0).nonzero()[:, 0]
    row, token = inverse[pair], pair // k
    if c["op"] == "dispatch":
        out = torch.zeros((T * k, d), dtype=torch.float64, device=DEV)
        out.index_copy_(0, row, s["x"].double()[token])
        return {"rows": out}
    rows = s["rows"].double().index_select(0, row)
    if c["op"] in ("dispatch_grad", "combine"):
        out = s["add"].double().clone() if "add" in s else \
            torch.zeros((T, d), dtype=torch.float64, device=DEV)
        if c["op"] == "combine":
            rows *= s["weights"].double().reshape(-1)[pair].unsqueeze(1)
        out.index_add_(0, token, rows)
        return {"y": out}
    dy = s["x"].double().index_select(0, token)
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[pair] = (dy * rows).sum(dim=1)
    out = torch.zeros((T * k, d), dtype=torch.float64, device=DEV)
    out[row] = dy * s["weights"].double().reshape(-1, 1)[pair]
    return {"drows": out, "dweights": dw.reshape(T, k)}


def _exact_kept(v, limit):
    out = torch.empty_like(v)
    for j in range(0, v.shape[1], 32):
        a = v[:, j:j + 32].abs()
        top = a.max(dim=1, keepdim=True)[0]
        unit = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top / 448.0, 1.0))))
        a = a / unit
        step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6) - 3)
        low = torch.floor(a / step) * step
        r = torch.round(a / step) * step
        if limit > 0:
            edge = limit / unit
            r = torch.where((a > edge) & (r <= edge), low + step, r)
            r = torch.where((a <= edge) & (r > edge), low, r)
        out[:, j:j + 32] = torch.copysign(r * unit, v[:, j:j + 32])
    return out


def _exact_experts(c, s):
    L, ends, train = s["layer"], s["ends"], c["op"] == "train"
    big = c["limit"] or math.inf
    zeros = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=DEV)
    out = {"y": zeros(s["x"])}
    if train:
        out["dx"] = zeros(s["x"])
        out.update({"d" + n: zeros(L[n]) for n in L})
    for e in range(c["experts"]):
        part = slice(ends[e], ends[e + 1])
        if ends[e] == ends[e + 1]:
            continue
        x = s["x"][part].double()
        wg, wu, wd = (L[n][e].double() for n in ("w_gate", "w_up", "w_down"))

        def halves(z, u):
            a, b = torch.minimum(z, torch.full_like(z, big)), u.clamp(min=-big, max=big)
            return a, b, 1 / (1 + torch.exp(-a))

        z, u = x.mm(wg.t()), x.mm(wu.t())
        a, b, q = halves(z, u)
        out["y"][part] = (a * b * q).mm(wd.t())
        if not train:
            continue
        if c["save"] == "mxfp8":
            z, u = _exact_kept(z, c["limit"]), _exact_kept(u, c["limit"])
            a, b, q = halves(z, u)
        dy = s["dy"][part].double()
        dh = dy.mm(wd)
        dz = torch.where(z > big, 0.0, dh * b * (q + a * q * (1 - q)))
        du = torch.where((u > big) | (u < -big), 0.0, dh * a * q)
        out["dx"][part] = dz.mm(wg) + du.mm(wu)
        out["dw_gate"][e] = dz.t().mm(x)
        out["dw_up"][e] = du.t().mm(x)
        out["dw_down"][e] = dy.t().mm(a * b * q)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "keep":
        return {"values": _exact_kept(s["src"].double(), case["limit"])}
    if case["op"] in ("experts", "train"):
        return _exact_experts(case, s)
    return _exact_sort(case, s)
