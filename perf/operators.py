"""What is timed of the operators: the MoE layer for a few tokens and the dense
product with bias, activation and residual, forward and with its gradient.

``own`` chooses between the plain torch form of each (32-bit arithmetic on the
same inputs) and the HIP kernels as a program calls them.
"""

import math

import torch

own = False

DEV = "cuda"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}

# Layer shapes of the package's named workloads and of its tests.
TINY = dict(dim=128, experts=16, topk=2, inter=64, groups=1, kept=1, score="softmax", scale=1.0,
            limit=0.0, route="learned", vocab=0, bias=False, kind="f32")
HASH = dict(dim=2048, experts=64, topk=4, inter=1024, groups=1, kept=1, score="softmax", scale=1.0,
            limit=0.0, route="hash", vocab=32768, bias=False, kind="bf16")
V3 = dict(dim=7168, experts=256, topk=8, inter=2048, groups=8, kept=4, score="sigmoid", scale=2.5,
          limit=0.0, route="learned", vocab=0, bias=True, kind="bf16")
FLASH = dict(dim=5120, experts=384, topk=8, inter=1536, groups=1, kept=1, score="sqrtsoftplus",
             scale=1.0, limit=10.0, route="learned", vocab=0, bias=True, kind="fp4")


def _few(name, shape, tokens, **change):
    return dict(shape, op="few", tokens=tokens, **change, name=name)


def _lin(name, op, rows, k, n, act, dtype="bf16", bias=True, residual=False, limit=0.0, pad=0):
    return dict(op=op, rows=rows, k=k, n=n, act=act, dtype=dtype, bias=bias, residual=residual,
                limit=limit, pad=pad, name=name)


def listed():
    return [
        # a test-sized fp32 layer: nothing but latency
        _few("few_tiny_f32_t3", TINY, 3),
        # hash-routed head layer, a handful of sequences decoding together
        _few("few_hash_bf16_t7", HASH, 7),
        # one user's next token through a large bf16 layer
        _few("few_v3_bf16_t1", V3, 1),
        # one user's next token through an FP4 layer
        _few("few_flash_fp4_t1", FLASH, 1),
        # a few drafted tokens of several users, FP4 experts on bf16 activations
        _few("few_flash_fp4_t5", FLASH, 5),
        # the largest batch of the decode form, MXFP8 activations on the FP4 experts
        _few("few_flash_mx_t16", FLASH, 16, kind="mx"),
        # one token through the gate|up of a dense layer: a weight stream
        _lin("linear_token_swiglu", "linear", 1, 7168, 2048, "swiglu"),
        # an fp32 model's layer at sizes nothing divides, rows inside a wider buffer
        _lin("linear_odd_f32", "linear", 203, 777, 1023, "gelu", dtype="f32", residual=True, pad=5),
        # down projection of a dense layer over a prompt, added to the residual stream
        _lin("linear_prompt_down", "linear", 4096, 2048, 7168, "none", residual=True),
        # a small fp32 training step
        _lin("train_small_f32", "train", 301, 256, 320, "silu", dtype="f32", residual=True),
        # gate|up of a dense layer in training at the hash workload's widths
        _lin("train_hash_width", "train", 4096, 2048, 1024, "swiglu", limit=10.0),
        # the same at the V4.1-Flash workload's widths and batch: the largest
        _lin("train_flash_width", "train", 8192, 5120, 1536, "swiglu", limit=10.0, bias=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        kind = rng.choice(["f32", "bf16", "bf16", "fp4", "fp4", "mx"])
        small = kind == "f32"
        unit = {"f32": 1, "bf16": 64, "fp4": 64, "mx": 128}[kind]
        dim = max(unit, _logint(rng, 64, 512 if small else 7168) // unit * unit)
        inter = max(unit, _logint(rng, 48, 256 if small else 2048) // unit * unit)
        groups = rng.choice([1, 1, 4, 8])
        experts = rng.choice([8, 16, 48, 64] if small else [8, 16, 64, 128, 256])
        if experts % (groups * 2) or groups * 2 > experts:
            groups = 1
        kept = rng.randint((groups + 1) // 2, groups)
        topk = rng.randint(1, min(8, experts // groups * kept))
        route = rng.choice(["learned", "learned", "hash"])
        if route == "hash":
            groups = kept = 1
        return dict(op="few", tokens=rng.randint(1, 16), dim=dim, experts=experts, topk=topk,
                    inter=inter, groups=groups, kept=kept,
                    score=rng.choice(["softmax", "sigmoid", "sqrtsoftplus"]),
                    scale=rng.choice([1.0, 2.5]), limit=rng.choice([0.0, 10.0]), route=route,
                    vocab=rng.randint(500, 40000) if route == "hash" else 0,
                    bias=route == "learned" and rng.random() < 0.5, kind=kind)
    op = rng.choice(["linear", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    top = 2048 if dtype == "f32" else 8192
    return dict(op=op, rows=_logint(rng, 1, top), k=_logint(rng, 16, min(top, 5120)),
                n=_logint(rng, 16, 1536 if op == "train" else min(top, 7168)),
                act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "swiglu"]),
                dtype=dtype, bias=rng.random() < 0.7, residual=rng.random() < 0.5,
                limit=rng.choice([0.0, 10.0]), pad=rng.choice([0, 0, 8, 3]))


# ---- inputs ----------------------------------------------------------------

def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + tag * 7919 + 17) % (1 << 62))
    return g


def _normal(shape, dtype, std, g):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _code_table():
    """256 E2M1 codes as often as a normal value quantised with its block's scale takes them."""
    mids = [0.125, 0.375, 0.625, 0.875, 1.25, 1.75, 2.5]        # in standard deviations
    cdf = [math.erf(m / math.sqrt(2.0)) for m in mids] + [1.0]
    table, at = [], 0
    for code, c in enumerate(cdf):
        upto = int(round(128 * c))
        table += [code] * (upto - at)
        at = upto
    return table + [t | 8 for t in table]


def _fp4(experts, n, k, g):
    """E2M1 codes [experts, n, k/2] and E8M0 scales [experts, n, k/32] of N(0, 1/k) weights."""
    table = torch.tensor(_code_table(), dtype=torch.uint8, device=DEV)
    codes = torch.empty((experts, n, k // 2), dtype=torch.uint8, device=DEV)
    for e in range(0, experts, 16):
        part = codes[e:e + 16]
        lo, hi = (table[torch.randint(0, 256, part.shape, device=DEV, generator=g,
                                      dtype=torch.int32)] for _ in range(2))
        part.copy_(lo | (hi << 4))
    top = 127 + math.floor(math.log2(2.2 / math.sqrt(k))) - 2
    scales = torch.empty((experts, n, k // 32), dtype=torch.uint8, device=DEV)
    scales.random_(0, 10, generator=g)
    scales.copy_(top - (scales < 3).to(torch.uint8))             # three blocks in ten one step lower
    return codes, scales


def _prepare_few(c, seed):
    T, d, E, k, I = c["tokens"], c["dim"], c["experts"], c["topk"], c["inter"]
    act = TDT["f32" if c["kind"] == "f32" else "bf16"]
    L = {"x": _normal((T, d), act, 1.0, _gen(seed, 1))}
    if c["route"] == "learned":
        L["gate_w"] = _normal((E, d), act, d ** -0.5, _gen(seed, 2))
        if c["bias"]:
            L["gate_bias"] = torch.empty(E, device=DEV).uniform_(-0.01, 0.01, generator=_gen(seed, 3))
    else:
        u = torch.rand((c["vocab"], E), device=DEV, generator=_gen(seed, 4))
        L["tid2eid"] = u.argsort(dim=1)[:, :k].to(torch.int32).contiguous()
        L["token_ids"] = torch.randint(0, c["vocab"], (T,), device=DEV, generator=_gen(seed, 5),
                                       dtype=torch.int32)
    for i, (m, n, kk) in enumerate((("gate", I, d), ("up", I, d), ("down", d, I))):
        if c["kind"] in ("fp4", "mx"):
            L["w_" + m], L["s_" + m] = _fp4(E, n, kk, _gen(seed, 10 + i))
        else:
            L["w_" + m] = _normal((E, n, kk), act, kk ** -0.5, _gen(seed, 10 + i))
        L["sh_" + m] = _normal((n, kk), act, kk ** -0.5, _gen(seed, 20 + i))
    s = {"case": c, "layer": L}
    if own:
        from mixture_experts_ffn_route_amd import binding, config
        low = c["kind"] in ("fp4", "mx")
        cfg = config.MoEConfig(
            dim=d, n_routed_experts=E, n_activated_experts=k, moe_inter_dim=I,
            n_expert_groups=c["groups"], n_limited_groups=c["kept"], score_func=c["score"],
            route_scale=c["scale"], swiglu_limit=c["limit"], route_mode=c["route"],
            vocab_size=c["vocab"], has_bias=c["bias"],
            act_dtype="f32" if c["kind"] == "f32" else "bf16",
            expert_dtype="fp4" if low else c["kind"],
            act_quant="mxfp8" if c["kind"] == "mx" else "none")
        s["B"] = binding
        s["cfg"], s["weights"] = binding.config_c(cfg), binding.weights_c(L)
        s["ws"] = binding.alloc_few_workspace(cfg, T)
        s["y"] = torch.empty_like(L["x"])
    return s


def _prepare_linear(c, seed):
    M, K, N, dt = c["rows"], c["k"], c["n"], TDT[c["dtype"]]
    two = c["act"] == "swiglu"

    def rows(width, tag):
        return _normal((M, width + c["pad"]), dt, 1.0, _gen(seed, tag))[:, :width]

    s = {"case": c, "x": rows(K, 1), "w": _normal((N, K), dt, K ** -0.5, _gen(seed, 2)),
         "w_up": _normal((N, K), dt, K ** -0.5, _gen(seed, 3)) if two else None,
         "bias": _normal((N,), dt, 0.1, _gen(seed, 4)) if c["bias"] else None,
         "bias_up": _normal((N,), dt, 0.1, _gen(seed, 5)) if c["bias"] and two else None,
         "residual": rows(N, 6) if c["residual"] else None}
    train = c["op"] == "train"
    if train:
        s["dy"] = rows(N, 7)
    if own:
        from mixture_experts_ffn_route_amd import binding, config
        cfg = config.LinearConfig(rows=M, in_dim=K, out_dim=N, dtype=c["dtype"],
                                  activation=c["act"], limit=c["limit"] if two else 0.0)
        s["B"], s["cfg"] = binding, cfg
        s["ws"] = binding.alloc_linear_workspace(cfg, backward=train)

        def like(t):
            return None if t is None else torch.empty(t.shape, dtype=t.dtype, device=DEV)

        s["y"] = torch.empty((M, N), dtype=dt, device=DEV)
        if train:
            keep = c["act"] != "none"
            s["z"] = torch.empty_like(s["y"]) if keep else None
            s["z_up"] = torch.empty_like(s["y"]) if two else None
            s["dx"] = torch.empty((M, K), dtype=dt, device=DEV)
            for n in ("w", "w_up", "bias", "bias_up"):
                s["d" + n] = like(s[n])
    return s


def prepare(case, seed):
    return _prepare_few(case, seed) if case["op"] == "few" else _prepare_linear(case, seed)


# ---- the plain forms -------------------------------------------------------

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _fp4_values(codes, scales):
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1)
    v = table[both.int()].reshape(codes.shape[0], -1, 32)
    return (v * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).reshape(codes.shape[0], -1)


def _mxfp8(v):
    """fp32 rows as the MXFP8 values that stand for them."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(dim=-1, keepdim=True)
    e = (torch.frexp(top)[1] - 9).clamp(-127, 127)
    unit = torch.exp2(torch.where(top > 0, e, torch.zeros_like(e)).float())
    q = (b / unit).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * unit).reshape(v.shape)


def _plain_swiglu(g, u, limit):
    if limit > 0:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g * torch.sigmoid(g) * u


def _plain_route(c, L):
    """Chosen experts [T, k] and their weights.  The scores in 64 bits: which
    expert comes in is decided on values next to one another."""
    k = c["topk"]
    if c["route"] == "hash":
        idx = L["tid2eid"][L["token_ids"].long()].long()
        return idx, torch.full(idx.shape, c["scale"] / k, device=DEV)
    z = L["x"].double() @ L["gate_w"].double().t()
    if c["score"] == "softmax":
        s = torch.exp(z - z.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    elif c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        s = torch.sqrt(z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
    key = s + L["gate_bias"].double() if c["bias"] else s
    G = c["groups"]
    if G > 1:
        by = key.reshape(key.shape[0], G, -1)
        top = by.sort(dim=2, descending=True)[0]
        rank = top[:, :, :2].sum(dim=2) if c["bias"] else top[:, :, 0]
        keep = rank.sort(dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        mask = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, keep, True)
        key = torch.where(mask.unsqueeze(2), by, -math.inf).reshape(key.shape)
    idx = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = s.gather(1, idx)
    if c["score"] != "softmax":
        w = w / w.sum(dim=1, keepdim=True)
    return idx, (w * c["scale"]).float()


def _plain_few(s):
    c, L = s["case"], s["layer"]
    idx, w = _plain_route(c, L)
    x = L["x"].float()
    xr = _mxfp8(x) if c["kind"] == "mx" else x

    def product(v, name, e):
        if c["kind"] in ("fp4", "mx"):
            m = _fp4_values(L["w_" + name][e], L["s_" + name][e])
        else:
            m = L["w_" + name][e].float()
        return v @ m.t()

    y = _plain_swiglu(x @ L["sh_gate"].float().t(), x @ L["sh_up"].float().t(), c["limit"])
    y = y @ L["sh_down"].float().t()
    for e in torch.unique(idx).tolist():
        hit = idx == e
        rows = hit.any(dim=1).nonzero()[:, 0]
        v = xr[rows]
        h = _plain_swiglu(product(v, "gate", e), product(v, "up", e), c["limit"])
        h = _mxfp8(h) if c["kind"] == "mx" else h
        y[rows] += (w * hit).sum(dim=1)[rows].unsqueeze(1) * product(h, "down", e)
    return y.to(L["x"].dtype)


def _act(z, name):
    """act(z) and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return (0.5 * z * (1 + t),
            0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z))


def _plain_linear(s):
    c = s["case"]
    x, w, dt = s["x"].float(), s["w"].float(), s["x"].dtype
    two = c["act"] == "swiglu"
    z = x @ w.t()
    z = z + s["bias"].float() if c["bias"] else z
    if two:
        w_up = s["w_up"].float()
        u = x @ w_up.t()
        u = u + s["bias_up"].float() if c["bias"] else u
        y = _plain_swiglu(z, u, c["limit"])
    else:
        y, slope = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    if c["op"] == "linear":
        return y.to(dt)
    dy = s["dy"].float()
    if two:
        top = c["limit"] if c["limit"] > 0 else math.inf
        g, v = z.clamp(max=top), u.clamp(-top, top)
        p = torch.sigmoid(g)
        dz = dy * v * p * (1 + g * (1 - p)) * (z <= top)
        du = dy * g * p * (u.abs() <= top)
        out = {"dx": dz @ w + du @ w_up, "dw_up": du.t() @ x}
        if c["bias"]:
            out["dbias_up"] = du.sum(dim=0)
    else:
        dz = dy * slope
        out = {"dx": dz @ w}
    out["dw"] = dz.t() @ x
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    out["y"] = y
    return {n: out[n].to(dt) for n in sorted(out)}


# ---- one pass --------------------------------------------------------------

def _own_few(s):
    s["B"].moe_forward_few(s["cfg"], s["weights"], s["layer"]["x"], s["layer"].get("token_ids"),
                           s["case"]["tokens"], s["y"], s["ws"])
    return s["y"]


def _own_linear(s):
    B, c = s["B"], s["case"]
    if c["op"] == "linear":
        B.moe_linear(s["cfg"], s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"],
                     w_up=s["w_up"], bias_up=s["bias_up"], ws=s["ws"])
        return s["y"]
    B.moe_linear(s["cfg"], s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"],
                 w_up=s["w_up"], bias_up=s["bias_up"], z=s["z"], z_up=s["z_up"], ws=s["ws"])
    B.moe_linear_backward(s["cfg"], s["dy"], s["x"], s["w"], w_up=s["w_up"], z=s["z"],
                          z_up=s["z_up"], dx=s["dx"], dw=s["dw"], dw_up=s["dw_up"],
                          dbias=s["dbias"], dbias_up=s["dbias_up"], ws=s["ws"])
    names = ("dbias", "dbias_up", "dw", "dw_up", "dx", "y")
    return {n: s[n] for n in names if s[n] is not None}


def run(state):
    if own:
        return (_own_few if state["case"]["op"] == "few" else _own_linear)(state)
    return (_plain_few if state["case"]["op"] == "few" else _plain_linear)(state)


def work(case):
    c = case
    if c["op"] == "few":
        T, d, E, k, I = c["tokens"], c["dim"], c["experts"], c["topk"], c["inter"]
        act = 4 if c["kind"] == "f32" else 2
        weight = {"f32": 4.0, "bf16": 2.0}.get(c["kind"], 0.5 + 1 / 32)
        touched = E * (1.0 - (1.0 - k / E) ** T)                 # distinct experts, expected
        learned = c["route"] == "learned"
        return {"bytes": int(3 * d * I * (touched * weight + act) + 2 * T * d * act +
                             (E * d * act if learned else 0)),
                "flops": 6 * d * I * T * (k + 1) + (2 * T * E * d if learned else 0)}
    M, K, N = c["rows"], c["k"], c["n"]
    size = 4 if c["dtype"] == "f32" else 2
    mats = 2 if c["act"] == "swiglu" else 1
    flops, items = 2 * M * N * K * mats, M * K + mats * N * K + M * N * (2 if c["residual"] else 1)
    if c["op"] == "train":
        # forward and backward as one path: x and the weights read once, dy read, y, dx and the
        # weights' gradients written
        flops *= 3
        items += M * N + M * K + mats * N * K
    return {"bytes": items * size, "flops": flops}


# ---- the definition in 64 bits ---------------------------------------------

def _exact_e4m3(v):
    """Nearest E4M3 value (ties to even), saturating at 448, by arithmetic."""
    a = v.abs()
    step = torch.exp2((torch.frexp(a)[1] - 1).clamp(min=-6).double() - 3.0)
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=448.0)


def _exact_mx(v):
    out = torch.zeros_like(v)
    for j in range(0, v.shape[1], 32):
        b = v[:, j:j + 32]
        top = b.abs().max(dim=1, keepdim=True)[0]
        unit = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 8.0)
        out[:, j:j + 32] = _exact_e4m3(b / unit) * unit
    return out


def _exact_matrix(c, L, name, e):
    if c["kind"] not in ("fp4", "mx"):
        return L["w_" + name][e].double()
    codes = L["w_" + name][e]
    full = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=DEV)
    for first, four in ((0, codes & 15), (1, codes >> 4)):
        m = (four & 7).double()
        mag = torch.where(m < 2, m * 0.5,
                          torch.exp2(torch.floor(m / 2) - 1) * (1 + 0.5 * torch.remainder(m, 2)))
        full[:, first::2] = torch.where(four >= 8, -mag, mag)
    return full * torch.exp2(L["s_" + name][e].double() - 127.0).repeat_interleave(32, dim=1)


def _exact_ffn(v, gate, up, limit):
    a, b = v @ gate.t(), v @ up.t()
    if limit > 0:
        a, b = torch.minimum(a, torch.full_like(a, limit)), b.clamp(-limit, limit)
    return a / (1.0 + torch.exp(-a)) * b


def _exact_few(c, L):
    T, E, k = c["tokens"], c["experts"], c["topk"]
    x = L["x"].double()
    G = torch.zeros((T, E), dtype=torch.float64, device=DEV)     # gate value of each expert
    if c["route"] == "hash":
        for t in range(T):
            for e in L["tid2eid"][int(L["token_ids"][t])].tolist():
                G[t, e] += c["scale"] / k
    else:
        z = (x @ L["gate_w"].double().t()).cpu()
        for t in range(T):
            if c["score"] == "softmax":
                s = torch.softmax(z[t], dim=0).tolist()
            elif c["score"] == "sigmoid":
                s = [1.0 / (1.0 + math.exp(-v)) for v in z[t].tolist()]
            else:
                s = [math.sqrt(max(v, 0.0) + math.log1p(math.exp(-abs(v)))) for v in z[t].tolist()]
            b = L["gate_bias"].tolist() if c["bias"] else [0.0] * E
            key = [p + q for p, q in zip(s, b)]
            size = E // c["groups"]
            score = []
            for g in range(c["groups"]):
                best = sorted(key[g * size:(g + 1) * size], reverse=True)
                score.append(sum(best[:2]) if c["bias"] else best[0])
            kept = sorted(range(c["groups"]), key=lambda g: (-score[g], g))[:c["kept"]]
            chosen = sorted((e for e in range(E) if e // size in kept), key=lambda e: (-key[e], e))[:k]
            total = 1.0 if c["score"] == "softmax" else sum(s[e] for e in chosen)
            for e in chosen:
                G[t, e] = s[e] / total * c["scale"]
    sh = [L["sh_" + n].double() for n in ("gate", "up", "down")]
    y = _exact_ffn(x, sh[0], sh[1], c["limit"]) @ sh[2].t()
    xr = _exact_mx(x) if c["kind"] == "mx" else x
    for e in G.any(dim=0).nonzero()[:, 0].tolist():
        t = G[:, e].nonzero()[:, 0]
        h = _exact_ffn(xr[t], _exact_matrix(c, L, "gate", e), _exact_matrix(c, L, "up", e), c["limit"])
        h = _exact_mx(h) if c["kind"] == "mx" else h
        y[t] += G[t, e].unsqueeze(1) * (h @ _exact_matrix(c, L, "down", e).t())
    return y


def _exact_linear(c, s):
    x, w = s["x"].double(), s["w"].double()
    z = x.mm(w.t()) + (s["bias"].double() if c["bias"] else 0.0)
    r = s["residual"].double() if c["residual"] else 0.0
    if c["act"] == "swiglu":
        top = c["limit"] or math.inf
        w_up = s["w_up"].double()
        u = x.mm(w_up.t()) + (s["bias_up"].double() if c["bias"] else 0.0)
        g, v = z.clamp(max=top), u.clamp(min=-top, max=top)
        e = torch.exp(-g)
        y = g * v / (1 + e) + r
        slope = v * (1 + e + g * e) / (1 + e) ** 2 * (z <= top)
        slope_up = g / (1 + e) * ((u <= top) & (u >= -top))
    else:
        name = c["act"]
        if name == "none":
            y, slope = z, torch.ones_like(z)
        elif name == "relu":
            y, slope = torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
        elif name == "silu":
            e = torch.exp(-z)
            y, slope = z / (1 + e), (1 + e + z * e) / (1 + e) ** 2
        elif name == "gelu":
            phi = torch.special.ndtr(z)
            y, slope = z * phi, phi + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
        else:
            q = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)   # 1 + tanh(q/2) = 2 sigmoid(q)
            p = 1 / (1 + torch.exp(-q))
            y = z * p
            slope = p + z * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)
        y = y + r
    if c["op"] == "linear":
        return y
    dy = s["dy"].double()
    dz = dy * slope
    out = {"y": y, "dx": dz.mm(w), "dw": dz.t().mm(x)}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    if c["act"] == "swiglu":
        du = dy * slope_up
        out["dx"] += du.mm(w_up)
        out["dw_up"] = du.t().mm(x)
        if c["bias"]:
            out["dbias_up"] = du.sum(0)
    return {n: out[n] for n in sorted(out)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_few(case, s["layer"]) if case["op"] == "few" else _exact_linear(case, s)
