"""Cases of the int8 products, the grouped products with 16-bit expert weights and their gradients, and
SiLU*mul with its gradient: sizes, inputs, plain forms and results in 64 bits.

A case's "kind" names the operator:
  linear_i8     activations quantized per token to 8-bit integers and multiplied by int8 weights with a scale per channel
  grouped_i8    the same with the weights of each row's expert (rows in expert order, ragged groups)
  grouped       products with 16-bit weights of each row's expert
  grouped_bwd   the gradients of that product with respect to its rows and its weights
  silu          h = silu(gate) * up of a stored gate_up result, and its gradient
"""
import torch

own = False
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a shared expert's down projection: the smallest call, latency alone
        dict(name="linear_i8_1", kind="linear_i8", T=1, N=2048, K=768, silu=False, x="bf16", out="bf16"),
        # a short prompt of odd length through a dense gate_up projection
        dict(name="linear_i8_77", kind="linear_i8", T=77, N=1536, K=2048, silu=True, x="f16", out="f16"),
        # a long prompt through the largest dense gate_up projection
        dict(name="linear_i8_4096", kind="linear_i8", T=4096, N=28672, K=4096, silu=True, x="bf16", out="bf16"),
        # a decode batch of 8 sequences, gate_up over 128 experts
        dict(name="grouped_i8_dec8", kind="grouped_i8", T=8, E=128, k=8, N=1536, K=2048, silu=True, gather=True, skew=0.0, x="bf16", out="bf16"),
        # a prompt of 800 tokens, the down projection over 256 experts
        dict(name="grouped_i8_800", kind="grouped_i8", T=800, E=256, k=8, N=2048, K=512, silu=False, gather=False, skew=0.0, x="bf16", out="f32"),
        # a large batch with uneven experts, some of them idle
        dict(name="grouped_i8_8192", kind="grouped_i8", T=8192, E=512, k=10, N=1024, K=2048, silu=True, gather=True, skew=0.5, x="bf16", out="bf16"),
        # a decode batch with unquantized experts
        dict(name="grouped_bf16_dec8", kind="grouped", T=8, E=128, k=8, N=1536, K=2048, silu=True, gather=True, skew=0.0, x="bf16", out="bf16"),
        # the down projection of eight large experts over a training batch
        dict(name="grouped_f16_4096", kind="grouped", T=4096, E=8, k=2, N=4096, K=14336, silu=False, gather=False, skew=0.3, x="f16", out="f32"),
        # gradients of a gate_up projection over many small experts
        dict(name="grouped_bwd_bf16_800", kind="grouped_bwd", T=800, E=256, k=8, N=1024, K=2048, gather=True, skew=0.3, x="bf16", out="bf16"),
        # gradients of a down projection over large experts, odd number of rows, weight gradients kept in 32 bits
        dict(name="grouped_bwd_f16_4095", kind="grouped_bwd", T=4095, E=8, k=2, N=4096, K=14336, gather=False, skew=0.3, x="f16", out="f32"),
        # a decode batch's activations
        dict(name="silu_512", kind="silu", R=512, I=768, x="bf16"),
        # a training batch's activations
        dict(name="silu_8192", kind="silu", R=8191, I=14336, x="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = round(lo * (hi / lo) ** rng.random() / step) * step
    return int(min(max(v, lo), hi))


def draw(rng):
    kind = rng.choice(["linear_i8", "grouped_i8", "grouped", "grouped_bwd", "silu"])
    if kind == "silu":
        return dict(kind=kind, R=_log(rng, 1, 8192), I=_log(rng, 64, 14336, 8), x=rng.choice(["bf16", "f16"]))
    while True:
        case = dict(kind=kind, x=rng.choice(["bf16", "f16"]))
        if kind == "linear_i8":
            case.update(T=_log(rng, 1, 4096), N=_log(rng, 64, 28672, 2), K=_log(rng, 256, 8192, 16))
        else:
            E = _log(rng, 4, 512)
            case.update(T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 10)), N=_log(rng, 128, 8192, 8), K=_log(rng, 256, 8192, 16),
                        gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.3, 0.5]))
        if kind != "grouped_bwd":
            case["silu"] = rng.random() < 0.5
        case["out"] = case["x"] if case.get("silu") else rng.choice([case["x"], "f32"])
        need = work(case)
        if need["bytes"] < 2.5e9 and need["flops"] < 9e11 and case.get("E", 1) * case["N"] * case["K"] < 6e8:
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


def _routing(gen, c):
    """Rows in expert order, as a permutation step leaves them: the expert offsets, each row's flat slot
    (token * k + slot), and the tables by which a plain form lays the groups out in equal blocks."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), generator=gen, device=DEVICE) + c["skew"] * torch.randn((1, E), generator=gen, device=DEVICE)
    ids = logits.topk(k, dim=1).indices.reshape(-1)
    rows = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEVICE)
    offsets[1:] = counts.cumsum(0)
    touched = torch.nonzero(counts).reshape(-1)
    most = int(counts.max())
    place = torch.arange(most, device=DEVICE)
    table = offsets[touched][:, None] + place  # [touched, most]: permuted row
    live = place < counts[touched][:, None]
    group = torch.repeat_interleave(torch.arange(len(touched), device=DEVICE), counts[touched])
    within = torch.arange(T * k, device=DEVICE) - offsets[touched][group]
    return dict(offsets=offsets.to(torch.int32), slots=rows.to(torch.int32), token=rows // k, touched=touched,
                table=torch.where(live, table, 0), live=live, group=group, within=within)


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = {"case": c}
    dt = TYPES[c["x"]]
    if c["kind"] == "silu":
        s["g"] = _rand(gen, (c["R"], 2 * c["I"]), dt)
        s["dh"] = _rand(gen, (c["R"], c["I"]), dt)
        return s
    N, K = c["N"], c["K"]
    if c["kind"] == "linear_i8":
        s["x"] = _rand(gen, (c["T"], K), dt)
        s["wq"] = _codes(gen, (N, K))
        s["ws"] = torch.rand(N, generator=gen, device=DEVICE).add_(0.5).mul_(1 / (35 * K ** 0.5))
        return s
    s.update(_routing(gen, c))
    R = c["T"] * c["k"]
    s["a"] = _rand(gen, (c["T"] if c["gather"] else R, K), dt)
    if c["kind"] == "grouped_i8":
        s["wq"] = _codes(gen, (c["E"], N, K))
        s["ws"] = torch.rand((c["E"], N), generator=gen, device=DEVICE).add_(0.5).mul_(1 / (35 * K ** 0.5))
        return s
    s["w"] = torch.empty((c["E"], N, K), dtype=dt, device=DEVICE)
    for e in range(c["E"]):
        s["w"][e] = _rand(gen, (N, K), dt, K ** -0.5)
    if c["kind"] == "grouped_bwd":
        s["dc"] = _rand(gen, (R, N), dt)
    return s


def _silu_mul(y):
    g, u = y.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _quantize(x):
    # the quotient next to a half needs more than 32 bits; scale and codes are those of 32-bit scales
    amax = x.abs().amax(dim=1, keepdim=True).double()
    s = (amax / 127).float()
    q = torch.round(x.double() / torch.where(s > 0, s, 1).double()).clamp_(-127, 127)
    return q.float(), s


def _all_or_some(t, touched):
    return t if len(touched) == t.shape[0] else t[touched]


def _blocks(s, rows, token=False):
    """[groups, most, cols]: each group's rows, 0 past its end."""
    at = s["table"] if not token else s["token"][s["table"]]
    return torch.where(s["live"][:, :, None], rows[at], 0)


def run(state):
    c = state["case"]
    out = TYPES[c["out"]] if "out" in c else None
    if own:
        return _run_own(state, c)
    if c["kind"] == "linear_i8":
        q, sx = _quantize(state["x"])
        y = (q @ state["wq"].float().t()) * (sx * state["ws"])
        return (_silu_mul(y) if c["silu"] else y).to(out)
    if c["kind"] == "silu":
        g, u = state["g"].float().chunk(2, dim=-1)
        dh, sg = state["dh"].float(), 1 / (1 + torch.exp(-g))
        dt = state["g"].dtype
        return {"h": (g * sg * u).to(dt), "dg": torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], dim=-1).to(dt)}
    touched, group, within = state["touched"], state["group"], state["within"]
    if c["kind"] == "grouped_i8":
        q, sx = _quantize(state["a"])
        w = _all_or_some(state["wq"], touched).float()
        y = torch.bmm(_blocks(state, q, c["gather"]), w.transpose(1, 2))[group, within]
        y = y * (sx[state["token"]] if c["gather"] else sx) * _all_or_some(state["ws"], touched)[group]
        return (_silu_mul(y) if c["silu"] else y).to(out)
    w = _all_or_some(state["w"], touched).float()
    a = _blocks(state, state["a"], c["gather"]).float()
    if c["kind"] == "grouped":
        y = torch.bmm(a, w.transpose(1, 2))[group, within]
        return (_silu_mul(y) if c["silu"] else y).to(out)
    dc = _blocks(state, state["dc"]).float()
    da = torch.bmm(dc, w)[group, within].to(state["a"].dtype)
    dw = torch.bmm(dc.transpose(1, 2), a).to(out)
    if len(touched) < c["E"]:
        whole = torch.zeros_like(state["w"], dtype=out)
        whole[touched] = dw
        dw = whole
    return {"da": da, "dw": dw}


def _run_own(s, c):
    import moe_w4a16_grouped_amd as moe

    epi = moe.MOE_EPI_SILU_MUL if c.get("silu") else moe.MOE_EPI_NONE
    out = {"bf16": moe.MOE_OUT_BF16, "f16": moe.MOE_OUT_F16, "f32": moe.MOE_OUT_F32}.get(c.get("out"))
    if c["kind"] == "linear_i8":
        return moe.moe_linear_i8(s["x"], s["wq"], s["ws"], epilogue=epi, out_dtype=out)
    if c["kind"] == "silu":
        return {"h": moe.moe_silu_mul(s["g"]), "dg": moe.moe_silu_mul_grad(s["g"], s["dh"])}
    slots, div = (s["slots"], c["k"]) if c["gather"] else (None, 1)
    if c["kind"] == "grouped_i8":
        q, sx = moe.moe_i8_quantize(s["a"])
        return moe.moe_grouped_gemm_i8(q, sx, slots, div, s["wq"], s["ws"], s["offsets"], len(s["slots"]), epilogue=epi, out_dtype=out)
    if c["kind"] == "grouped":
        return moe.moe_grouped_gemm_w16(s["a"], slots, div, s["w"], s["offsets"], len(s["slots"]), epilogue=epi, out_dtype=out)
    return {"da": moe.moe_grouped_gemm_w16_dx(s["dc"], s["w"], s["offsets"]),
            "dw": moe.moe_grouped_gemm_w16_dw(s["dc"], s["a"], slots, div, s["offsets"], out_dtype=out)}


def work(case):
    c = case
    if c["kind"] == "silu":  # h: read gate and up, write h; gradient: read gate, up and dh, write both gradients
        n = c["R"] * c["I"]
        return {"bytes": 2 * n * (3 + 5), "flops": 20 * n}
    N, K, T = c["N"], c["K"], c["T"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    cols = N // 2 if c.get("silu") else N
    if c["kind"] == "linear_i8":
        return {"bytes": T * K * 2 + N * K + N * 4 + T * cols * size[c["out"]], "flops": 2 * T * N * K}
    E, R = c["E"], T * c["k"]
    touched = E * (1 - (1 - c["k"] / E) ** T)  # experts with a row, of even routing
    rows = T if c["gather"] else R
    if c["kind"] == "grouped_i8":
        return {"bytes": int(rows * K * 2 + touched * (N * K + N * 4) + R * cols * size[c["out"]]), "flops": 2 * R * N * K}
    if c["kind"] == "grouped":
        return {"bytes": int(rows * K * 2 + touched * N * K * 2 + R * cols * size[c["out"]]), "flops": 2 * R * N * K}
    return {"bytes": int(R * N * 2 + rows * K * 2 + touched * N * K * 2 + R * K * 2 + E * N * K * size[c["out"]]), "flops": 4 * R * N * K}


def _exact_rows(x):
    x = x.double()
    s = (x.abs().max(dim=1).values / 127).float().double()[:, None]
    return torch.where(s > 0, torch.clamp(torch.round(x / s), -127, 127), 0) * s


def _exact_epilogue(c, y):
    if not c["silu"]:
        return y
    half = y.shape[1] // 2
    return y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "silu":
        z = s["g"].double()
        g, u = z[:, :c["I"]], z[:, c["I"]:]
        sg, d = torch.sigmoid(g), s["dh"].double()
        return {"h": g * sg * u, "dg": torch.cat([d * u * (sg + g * sg * (1 - sg)), d * g * sg], dim=1)}
    if c["kind"] == "linear_i8":
        w = s["wq"].double() * s["ws"].double()[:, None]
        return _exact_epilogue(c, torch.mm(_exact_rows(s["x"]), w.t()))
    ends = s["offsets"].tolist()
    a = _exact_rows(s["a"]) if c["kind"] == "grouped_i8" else s["a"].double()
    if c["gather"]:
        a = a[s["slots"].long() // c["k"]]
    parts, grads = [], []
    if c["kind"] == "grouped_bwd":
        grads = torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float64, device=DEVICE)
    for e in range(c["E"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        if c["kind"] == "grouped_i8":
            w = s["wq"][e].double() * s["ws"][e].double()[:, None]
        else:
            w = s["w"][e].double()
        if c["kind"] == "grouped_bwd":
            d = s["dc"][lo:hi].double()
            parts.append(torch.mm(d, w))
            grads[e] = torch.mm(d.t(), a[lo:hi])
        else:
            parts.append(_exact_epilogue(c, torch.mm(a[lo:hi], w.t())))
    rows = torch.cat(parts)
    return {"da": rows, "dw": grads} if c["kind"] == "grouped_bwd" else rows
