"""Cases of the root-mean-square norm with the residual's addition, its gradient, and the whole expert layer for a
few tokens: sizes, inputs, plain forms and results in 64 bits.

A case's "kind" names the operator:
  norm       s = x + residual, y = s / rms(s) * w, with 8-bit codes and scales of y (int8 per row, FP8 per 128 columns)
  norm_grad  the gradients of that norm with respect to its input and its weight
  few_w16    the expert layer (routing, gate_up, SiLU*mul, down, weighted sum) of up to 16 tokens, bf16 weights
  few_w8a16  the same with int8 weights and a scale per channel
"""
import torch

own = False
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token in front of its experts: 16 bits for the router, int8 for the products
        dict(name="norm_1", kind="norm", T=1, H=2048, x="bf16", w="bf16", residual=True, y=True, quant="i8", eps=1e-6),
        # a prompt of odd length, fp32 weight, int8 alone
        dict(name="norm_801", kind="norm", T=801, H=2048, x="f16", w="f32", residual=False, y=False, quant="i8", eps=1e-5),
        # a long prompt: 16 bits for the router and FP8 for the experts
        dict(name="norm_8191", kind="norm", T=8191, H=4096, x="bf16", w="bf16", residual=True, y=True, quant="f8", eps=1e-6),
        # gradients of a short sequence, fp32 weight
        dict(name="norm_grad_77", kind="norm_grad", T=77, H=2048, x="f16", w="f32", residual=False, eps=1e-5),
        # gradients of a training batch, the residual stream's gradient added
        dict(name="norm_grad_8191", kind="norm_grad", T=8191, H=4096, x="bf16", w="bf16", residual=True, eps=1e-6),
        # one token through unquantized experts
        dict(name="few_w16_1", kind="few_w16", T=1, E=128, k=8, H=2048, I=768),
        # a decode batch of 8 sequences
        dict(name="few_w16_8", kind="few_w16", T=8, E=128, k=8, H=2048, I=768),
        # 16 sequences over eight large experts, all of them read
        dict(name="few_w16_large", kind="few_w16", T=16, E=8, k=2, H=4096, I=14336),
        # one token through int8 experts
        dict(name="few_w8_1", kind="few_w8a16", T=1, E=128, k=8, H=2048, I=768),
        # sizes that fill no whole tile
        dict(name="few_w8_odd", kind="few_w8a16", T=11, E=60, k=6, H=1040, I=336),
        # the largest batch over many experts
        dict(name="few_w8_16", kind="few_w8a16", T=16, E=256, k=8, H=2048, I=512),
    ]


def _log(rng, lo, hi, step=1):
    v = round(lo * (hi / lo) ** rng.random() / step) * step
    return int(min(max(v, lo), hi))


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "few_w16", "few_w8a16"])
    if kind in ("norm", "norm_grad"):
        x = rng.choice(["bf16", "f16"])
        case = dict(kind=kind, x=x, w=rng.choice([x, "f32"]), residual=rng.random() < 0.5, eps=rng.choice([1e-6, 1e-5]))
        quant = rng.choice(["none", "i8", "f8"]) if kind == "norm" else "none"
        case.update(T=_log(rng, 1, 8192), H=_log(rng, 128, 8192, {"none": 8, "i8": 16, "f8": 128}[quant]))
        if kind == "norm":
            case.update(quant=quant, y=quant == "none" or rng.random() < 0.5)
        return case if work(case)["bytes"] < 3.2e8 else draw(rng)
    while True:
        E = _log(rng, 4, 512)
        case = dict(kind=kind, T=_log(rng, 1, 16), E=E, k=rng.randint(1, min(E, 10)), H=_log(rng, 128, 8192, 16),
                    I=_log(rng, 64, 14336, 16))
        if case["T"] * case["H"] <= 65536 and work(case)["bytes"] < 2.5e9 and 3 * E * case["H"] * case["I"] < 2e9:
            return case


def _rand(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).mul_(scale).to(dtype)


def _codes(gen, shape):
    # weights of normal distribution whose largest magnitude of a channel has the code 127
    out = torch.empty(shape, dtype=torch.int8, device=DEVICE)
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 26) // shape[-1])
    for at in range(0, flat.shape[0], step):
        part = flat[at:at + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEVICE).mul_(35.0).round_().clamp_(-127, 127))
    return out


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = {"case": c}
    if c["kind"] in ("norm", "norm_grad"):
        dt, T, H = TYPES[c["x"]], c["T"], c["H"]
        s["w"] = torch.rand(H, generator=gen, device=DEVICE).add_(0.5).to(TYPES[c["w"]])
        # a few channels of a residual stream are much larger than the others
        channel = torch.ones(H, device=DEVICE)
        channel[torch.randint(0, H, (max(1, H // 512),), generator=gen, device=DEVICE)] = 20.0
        if c["kind"] == "norm":
            s["x"] = (_rand(gen, (T, H), torch.float32) * (1 if c["residual"] else channel)).to(dt)
            s["r"] = (_rand(gen, (T, H), torch.float32, 3.0) * channel).to(dt) if c["residual"] else None
        else:
            s["s"] = (_rand(gen, (T, H), torch.float32, 3.0) * channel).to(dt)
            s["dy"] = _rand(gen, (T, H), dt)
            s["ds"] = _rand(gen, (T, H), dt) if c["residual"] else None
        return s
    T, E, H, I = c["T"], c["E"], c["H"], c["I"]
    s["x"] = _rand(gen, (T, H), torch.bfloat16)
    s["logits"] = _rand(gen, (T, E), torch.float32)
    s["ids"] = torch.empty((T, c["k"]), dtype=torch.int32, device=DEVICE)  # a program's own buffers for the routing
    s["weight"] = torch.empty((T, c["k"]), device=DEVICE)
    if c["kind"] == "few_w16":
        s["w13"] = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=DEVICE)
        s["w2"] = torch.empty((E, H, I), dtype=torch.bfloat16, device=DEVICE)
        for e in range(E):
            s["w13"][e] = _rand(gen, (2 * I, H), torch.bfloat16, H ** -0.5)
            s["w2"][e] = _rand(gen, (H, I), torch.bfloat16, I ** -0.5)
    else:
        s["w13"] = _codes(gen, (E, 2 * I, H))
        s["w2"] = _codes(gen, (E, H, I))
        s["w13_s"] = torch.rand((E, 2 * I), generator=gen, device=DEVICE).add_(0.5).mul_(1 / (35 * H ** 0.5))
        s["w2_s"] = torch.rand((E, H), generator=gen, device=DEVICE).add_(0.5).mul_(1 / (35 * I ** 0.5))
    return s


def _e4m3(v):
    """The nearest E4M3 values, ties to even: 3 bits behind the leading one, the least step 2^-9."""
    steps = torch.tensor([2.0 ** n for n in range(-9, 7)], dtype=v.dtype, device=v.device)
    _, e = torch.frexp(v)
    step = steps[(e + 5).clamp_min(0)]
    return torch.round(v / step) * step


def _plain_norm(state, c):
    s = state["x"].float()
    out = {}
    if state["r"] is not None:
        s = (s + state["r"].float()).to(state["x"].dtype)
        out["s"] = s
        s = s.float()
    w = state["w"].float()
    rstd = 1 / torch.sqrt((s * s).sum(dim=1, keepdim=True) / c["H"] + c["eps"])
    if c["y"]:
        out["y"] = (s * rstd * w).to(state["x"].dtype)
    if c["quant"] != "none":
        z = s.double() * w.double()  # the quotient next to a border needs more than 32 bits
        if c["quant"] == "f8":
            z = z.view(c["T"], -1, 128)
        else:
            z = z.view(c["T"], 1, c["H"])
        top = 127.0 if c["quant"] == "i8" else 448.0
        amax = z.abs().amax(dim=2, keepdim=True)
        v = z * top / torch.where(amax > 0, amax, 1.0)
        code = torch.round(v).to(torch.int8) if c["quant"] == "i8" else _e4m3(v).to(torch.float8_e4m3fn)
        out["q"] = code.view(c["T"], c["H"])
        out["q_scale"] = (amax * rstd.double().view(-1, 1, 1) / top).float().view(c["T"], -1)
    return out


def _plain_norm_grad(state, c):
    s, dy, w = state["s"].float(), state["dy"].float(), state["w"].float()
    rstd = 1 / torch.sqrt((s * s).sum(dim=1, keepdim=True) / c["H"] + c["eps"])
    xhat = s * rstd
    g = dy * w
    dx = rstd * (g - xhat * ((g * xhat).sum(dim=1, keepdim=True) / c["H"]))
    if state["ds"] is not None:
        dx = dx + state["ds"].float()
    return {"dx": dx.to(state["s"].dtype), "dw": (dy * xhat).sum(dim=0).to(state["w"].dtype)}


def _route(logits, k):
    # equal logits in the order of their experts
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.exp(top[:, :k] - top[:, :1])
    return ids[:, :k], p / p.sum(dim=1, keepdim=True)


def _plain_layer(state, rows, of):
    """rows [n, m, H] through the experts `of` (None: all of them, n = E): [n, m, H]."""
    some = (lambda t: t.float()) if of is None else (lambda t: t[of].float())
    g = torch.bmm(rows, some(state["w13"]).transpose(1, 2))
    if "w13_s" in state:
        g = g * some(state["w13_s"])[:, None]
    gate, up = g.chunk(2, dim=2)
    o = torch.bmm(gate / (1 + torch.exp(-gate)) * up, some(state["w2"]).transpose(1, 2))
    return o * some(state["w2_s"])[:, None] if "w2_s" in state else o


def _plain_few(state, c):
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    ids, weight = _route(state["logits"], k)
    x = state["x"].float()
    if T * k < E:  # the weights of each row's expert
        rows = x[:, None].expand(T, k, H).reshape(T * k, 1, H)
        y = (_plain_layer(state, rows, ids.reshape(-1)).view(T, k, H) * weight[:, :, None]).sum(dim=1)
    else:  # every token through every expert, those that it did not choose with the weight 0
        share = torch.zeros((T, E), device=DEVICE).scatter_(1, ids, weight)
        y = (_plain_layer(state, x.expand(E, T, H), None) * share.t()[:, :, None]).sum(dim=0)
    return {"y": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weight": weight}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["kind"] == "norm":
        return _plain_norm(state, c)
    if c["kind"] == "norm_grad":
        return _plain_norm_grad(state, c)
    return _plain_few(state, c)


def _run_own(s, c):
    import moe_w4a16_grouped_amd as moe

    if c["kind"] == "norm":
        quant = {"none": moe.MOE_QUANT_NONE, "i8": moe.MOE_QUANT_I8, "f8": moe.MOE_QUANT_F8}[c["quant"]]
        res, y, q, q_scale = moe.moe_rmsnorm_add(s["x"], s["w"], c["eps"], residual=s["r"], quant=quant, want_y=c["y"])
        if c["quant"] == "f8":
            q = q.view(torch.float8_e4m3fn)
        out = {"s": res, "y": y, "q": q, "q_scale": None if q is None else q_scale.view(c["T"], -1)}
        return {name: t for name, t in out.items() if t is not None}
    if c["kind"] == "norm_grad":
        dx, dw = moe.moe_rmsnorm_add_grad(s["dy"], s["s"], s["w"], c["eps"], ds=s["ds"])
        return {"dx": dx, "dw": dw}
    ids, weight = s["ids"], s["weight"]
    if c["kind"] == "few_w16":
        y = moe.moe_ffn_few_w16(s["x"], s["logits"], s["w13"], s["w2"], c["k"], topk_ids_out=ids, topk_w_out=weight)
    else:
        y = moe.moe_ffn_few_w8a16(s["x"], s["logits"], s["w13"], s["w13_s"], s["w2"], s["w2_s"], c["k"], topk_ids_out=ids,
                                  topk_w_out=weight)
    return {"y": y, "ids": ids, "weight": weight}


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    T, H = c["T"], c["H"]
    if c["kind"] == "norm":
        # read x (and the residual), write the sum, the normalised row and its codes with their scales
        row = 2 + 4 * c["residual"] + 2 * c["y"] + (c["quant"] != "none")
        scales = {"none": 0, "i8": 1, "f8": H // 128}[c["quant"]]
        return {"bytes": T * H * row + T * scales * 4 + H * size[c["w"]], "flops": T * H * 6}
    if c["kind"] == "norm_grad":
        return {"bytes": T * H * (6 + 2 * c["residual"]) + 2 * H * size[c["w"]], "flops": T * H * 10}
    E, k, I = c["E"], c["k"], c["I"]
    touched = E * (1 - (1 - k / E) ** T)  # experts that a token chose, of even routing
    weights = 3 * I * H * 2 if c["kind"] == "few_w16" else 3 * I * H + (2 * I + H) * 4
    return {"bytes": int(touched * weights + T * (E * 4 + H * 4 + k * 8)), "flops": 6 * T * k * I * H}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "norm":
        return _exact_norm(c, s)
    if c["kind"] == "norm_grad":
        return _exact_norm_grad(c, s)
    return _exact_few(c, s)


def _exact_norm(c, s):
    v = s["x"].double()
    out = {"s": None, "y": None, "q": None, "q_scale": None}
    if s["r"] is None:
        del out["s"]
    else:
        v = (v + s["r"].double()).to(s["x"].dtype).double()
        out["s"] = v
    y = v / torch.sqrt(torch.mean(v ** 2, dim=1) + c["eps"])[:, None] * s["w"].double()
    if c["y"]:
        out["y"] = y
    else:
        del out["y"]
    if c["quant"] == "none":
        del out["q"], out["q_scale"]
    elif c["quant"] == "i8":
        z = v * s["w"].double()  # a row's codes do not depend on its norm
        most = torch.max(z.abs(), dim=1).values[:, None]
        out["q"] = torch.where(most > 0, (z * 127 / most).round(), 0).to(torch.int8)
        out["q_scale"] = torch.max(y.abs(), dim=1).values[:, None] / 127
    else:
        z = (v * s["w"].double()).reshape(-1, 128)
        most = torch.max(z.abs(), dim=1).values[:, None]
        v = torch.where(most > 0, z * 448 / most, 0)
        power = (v.view(torch.int64) & (0x7FF << 52)).view(torch.float64)  # the power of two at or below |v|
        unit = power.clamp_min(2.0 ** -6) / 8
        out["q"] = ((v / unit).round() * unit).reshape(c["T"], c["H"])
        out["q_scale"] = torch.max(y.abs().reshape(c["T"], -1, 128), dim=2).values / 448
    return out


def _exact_norm_grad(c, s):
    v, d, w = s["s"].double(), s["dy"].double(), s["w"].double()
    scale = torch.rsqrt(torch.mean(v ** 2, dim=1) + c["eps"])[:, None]
    dw = torch.sum(d * v * scale, dim=0)
    dx = scale * d * w - v * scale ** 3 * torch.mean(d * w * v, dim=1)[:, None]
    return {"dx": dx if s["ds"] is None else dx + s["ds"].double(), "dw": dw}


def _exact_few(c, s):
    T, k = c["T"], c["k"]
    logits = s["logits"].double()
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    weight = torch.softmax(torch.gather(logits, 1, ids), dim=1)
    y = torch.zeros((T, c["H"]), dtype=torch.float64, device=DEVICE)
    for e in torch.unique(ids).tolist():
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        up = s["w13"][e].double()
        down = s["w2"][e].double()
        if "w2_s" in s:
            up, down = up * s["w13_s"][e].double()[:, None], down * s["w2_s"][e].double()[:, None]
        g, u = torch.mm(s["x"][t].double(), up.t()).split(c["I"], dim=1)
        y[t] += torch.mm(g * torch.sigmoid(g) * u, down.t()) * weight[t, slot][:, None]
    return {"y": y, "ids": ids.to(torch.int32), "weight": weight}
