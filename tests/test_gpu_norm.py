"""The root-mean-square norm with the residual's addition, its 8-bit outputs and its gradient, against plain forms in 64
bits, at the sizes and values where they can go wrong.

Bounds.  Squares (exact in fp32, of 16-bit values) are added by fours in fp32, three roundings of 2^-24 of positive sums, and
those sums in 64 bits: the mean is off by 3 * 2^-24, its inverse root by half of that.  y = (s * r) * w in fp32: r 1.5 * 2^-24 and
2^-24 for its own rounding, the two products 2^-24 each: 4.6 * 2^-24 in all, then half a step of the type.  A scale is a
64-bit product with that root, rounded once: 2.6 * 2^-24.  Codes are those of the real quotient: equal."""
import pytest
import torch

import moe_w4a16_grouped_amd as moe
from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NONE, I8, F8 = moe.MOE_QUANT_NONE, moe.MOE_QUANT_I8, moe.MOE_QUANT_F8
U = 2.0 ** -24


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _weight(H, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(H, generator=g, device="cuda") + 0.5).to(dtype)


def _e4m3(v):
    """Nearest E4M3 value of each double, ties to even."""
    power = (v.view(torch.int64) & (0x7FF << 52)).view(torch.float64)
    unit = power.clamp_min(2.0 ** -6) / 8
    return torch.round(v / unit) * unit


def _reference(x, r, w, eps, quant):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    v, wd = s.double(), w.double()
    rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)
    y = v * rstd * wd
    if quant == NONE:
        return s, y, None, None
    z = v * wd
    z = z.view(x.shape[0], 1, -1) if quant == I8 else z.view(x.shape[0], -1, 128)
    top = 127.0 if quant == I8 else 448.0
    most = z.abs().amax(dim=2, keepdim=True)
    quotient = torch.where(most > 0, z * top / torch.where(most > 0, most, 1.0), 0.0)
    scale = most * rstd[:, :, None] / top
    codes = torch.where(scale.float() > 0, torch.round(quotient) if quant == I8 else _e4m3(quotient), 0.0)
    return s, y, codes.view(x.shape), scale.squeeze(2)


def _check(x, r, w, eps, quant, want_y, got):
    s, y, codes, scale = _reference(x, r, w, eps, quant)
    if r is None:
        assert got[0] is None
    else:
        assert torch.equal(got[0], s)
    if want_y:
        ru.assert_close(got[1], y, 4.6 * U * y.abs(), "y")
    else:
        assert got[1] is None
    if quant == NONE:
        assert got[2] is None and got[3] is None
        return
    if quant == I8:
        scale = scale[:, 0]
    assert got[3].shape == scale.shape
    assert bool(((got[3].double() - scale).abs() <= scale * U * 2.6 + 2.0 ** -149).all())
    q = got[2].double() if quant == I8 else got[2].view(torch.float8_e4m3fn).double()
    assert torch.equal(q, codes)


SIZES = [(1, 8), (3, 16), (5, 128), (4, 512), (7, 640), (2, 1048), (77, 2048), (1, 2048), (3, 2304), (9, 4096), (2, 4104), (5, 8192),
         (2, 8448), (3, 16384), (600, 128)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("x_dtype,w_dtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("quant,want_y", [(NONE, True), (I8, True), (I8, False), (F8, True), (F8, False)])
def test_norm(T, H, x_dtype, w_dtype, quant, want_y):
    if H % {NONE: 8, I8: 16, F8: 128}[quant]:
        pytest.skip("not a size of this quantization")
    x, r, w = _rand((T, H), x_dtype, T + H), _rand((T, H), x_dtype, T + H + 1, 3.0), _weight(H, w_dtype, H)
    for residual in (None, r):
        got = moe.moe_rmsnorm_add(x, w, 1e-5, residual=residual, quant=quant, want_y=want_y)
        _check(x, residual, w, 1e-5, quant, want_y, got)


@pytest.mark.parametrize("H,quant", [(520, NONE), (528, I8), (768, I8), (640, F8), (1024, F8), (1024, NONE)])
def test_many_short_rows(H, quant):
    """Rows enough that a wave takes each, of ordinary and of far magnitudes."""
    T = 2050
    x, r, w = _rand((T, H), BF16, 1), _rand((T, H), BF16, 2), _weight(H, BF16, 3)
    for at, f in ((0, 1e30), (5, 1e-36), (1027, 1e20), (T - 1, 0.0)):
        x[at] *= f
        r[at] *= f
    for residual in (None, r):
        _check(x, residual, w, 1e-5, quant, True, moe.moe_rmsnorm_add(x, w, 1e-5, residual=residual, quant=quant))


def test_int8_ties():
    """Quotients on and next to a half: the largest product is 127 * 2^6, so that 127 z / max is z / 64, and weights in fp32
    move a product by its last bit to either side."""
    H = 1024
    z = (torch.arange(H, device="cuda") % 254 - 127).double() + 0.5
    x = torch.full((3, H), 1.0, device="cuda", dtype=F16)
    w = (z * 64).float()
    w[0] = 127.0 * 64
    up, down = torch.nextafter(w, torch.full_like(w, 1e9)), torch.nextafter(w, torch.full_like(w, -1e9))
    up[0] = down[0] = w[0]
    for weight in (w, up, down):
        weight = torch.where(weight.abs() > 127 * 64, torch.zeros_like(weight), weight)
        _check(x, None, weight, 1e-6, I8, True, moe.moe_rmsnorm_add(x, weight, 1e-6, quant=I8))


def test_int8_ties_of_sixteen_bits():
    """Rows of every bf16 significand over each largest value: many quotients are exact halves."""
    v = torch.arange(128, 256, device="cuda", dtype=F32)
    x = torch.cat([v, v / 2, v / 4, -v / 8, v / 16, v / 32, v / 64, torch.zeros(128, device="cuda")]).to(BF16).repeat(128, 1)
    x[:, -1] = torch.arange(256, 512, 2, device="cuda").to(BF16)
    w = torch.ones(x.shape[1], dtype=BF16, device="cuda")
    for quant in (I8, F8):
        _check(x, None, w, 1e-6, quant, True, moe.moe_rmsnorm_add(x, w, 1e-6, quant=quant))


def test_fp8_borders():
    """Blocks whose largest value is 448: every border between two E4M3 values, subnormal ones too, and its neighbours by
    the last bit of an fp32 weight."""
    codes = torch.arange(0, 127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    border = (codes[:-1] + codes[1:]) / 2
    for to in (0.0, 1e9, -1e9):
        for sign in (1.0, -1.0):
            w = torch.zeros((2, 128), device="cuda")
            w[0, :63], w[1, :63] = (sign * border[:63]).float(), (sign * border[63:126]).float()
            if to:
                w = torch.where(w != 0, torch.nextafter(w, torch.full_like(w, to)), w)
            w[:, 127] = 448.0
            w = w.reshape(-1)
            x = torch.ones((2, 256), dtype=BF16, device="cuda")
            _check(x, None, w, 1e-6, F8, True, moe.moe_rmsnorm_add(x, w, 1e-6, quant=F8))


@pytest.mark.parametrize("quant", [NONE, I8, F8])
@pytest.mark.parametrize("value", [1e-38, 2.0 ** -130, 3e38, 1e20])
def test_far_magnitudes(quant, value):
    """Squares that fp32 cannot hold, products that pass it, and scales of tiny rows."""
    x, w = _rand((4, 256), F32, 5).clamp(-1, 1).mul(value).to(BF16), _weight(256, F32, 6) * 2
    x[1] = 0
    got = moe.moe_rmsnorm_add(x, w, 1e-6, quant=quant)
    _check(x, None, w, 1e-6, quant, True, got)
    tiny = (_rand((4, 256), F32, 5) * 2.0 ** -120).to(BF16)  # r = 2^60 with an eps as small
    _check(tiny, None, w, 2.0 ** -120, quant, True, moe.moe_rmsnorm_add(tiny, w, 2.0 ** -120, quant=quant))


@pytest.mark.parametrize("w_dtype", [BF16, F32])
@pytest.mark.parametrize("quant", [I8, F8])
def test_blocks_of_far_magnitudes_in_one_row(quant, w_dtype):
    """Blocks whose products vanish in fp32, or nearly, beside ordinary ones; blocks and rows of zeros."""
    H = 1024
    x = _rand((5, H), F32, 3)
    scale = torch.tensor([1.0, 2.0 ** -40, 2.0 ** -100, 2.0 ** -120, 0.0, 2.0 ** 30, 2.0 ** -62, 1e-3], device="cuda").repeat_interleave(128)
    x[:3] *= scale
    x[2] *= 2.0 ** -20
    x[3] = 0
    w = _weight(H, F32, 4)
    w[256:512] *= 2.0 ** -35
    x, w = x.to(BF16), w.to(w_dtype)
    for eps in (1e-6, 1e-30):
        _check(x, None, w, eps, quant, True, moe.moe_rmsnorm_add(x, w, eps, quant=quant))


@pytest.mark.parametrize("quant", [I8, F8])
def test_rows_without_finite_values(quant):
    """An infinity or a NaN reaches its own row alone, whose scales are NaN and whose codes are 0."""
    x, w = _rand((6, 512), BF16, 9), _weight(512, BF16, 8)
    plain = moe.moe_rmsnorm_add(x, w, 1e-6, quant=quant)
    x[1, 3], x[4, 200] = float("inf"), float("nan")
    s, y, q, scale = moe.moe_rmsnorm_add(x, w, 1e-6, quant=quant)
    rows = torch.tensor([0, 2, 3, 5], device="cuda")
    for a, b in ((y, plain[1]), (q, plain[2]), (scale, plain[3])):
        assert torch.equal(a[rows], b[rows])
    assert bool(scale[[1, 4]].isnan().all()) and not bool(q[[1, 4]].any())
    assert bool(y[1, 3].isnan()) and not bool(y[1, :3].any()) and bool(y[4].isnan().all())
    w[7] = float("nan")
    _, y, q, scale = moe.moe_rmsnorm_add(plain[1], w, 1e-6, quant=quant)
    assert bool(scale.isnan().all()) and not bool(q.any()) and bool(y[:, 7].isnan().all()) and not bool(y[:, 8:].isnan().any())


def test_in_place_and_rows_behind():
    T, H = 5, 2048
    x, r, w = _rand((T + 2, H), BF16, 1), _rand((T + 2, H), BF16, 2), _weight(H, BF16, 3)
    ref = moe.moe_rmsnorm_add(x[:T], w, 1e-6, residual=r[:T], quant=I8)
    for target in ("x", "residual"):
        a, b = x.clone(), r.clone()
        s = a if target == "x" else b
        y = b if target == "x" else a
        q = torch.full((T + 2, H), 77, dtype=torch.int8, device="cuda")
        scale = torch.full((T + 2,), 7.0, device="cuda")
        behind = s[T:].clone(), y[T:].clone()
        moe.moe_rmsnorm_add(a[:T], w, 1e-6, residual=b[:T], quant=I8, s=s[:T], y=y[:T], q=q[:T], q_scale=scale[:T])
        for got, want in zip((s, y, q, scale), ref):
            assert torch.equal(got[:T], want)
        assert torch.equal(s[T:], behind[0]) and torch.equal(y[T:], behind[1])
        assert bool((q[T:] == 77).all()) and bool((scale[T:] == 7.0).all())


def test_no_rows_and_many():
    w = _weight(256, BF16, 1)
    s, y, q, scale = moe.moe_rmsnorm_add(_rand((0, 256), BF16, 1), w, 1e-6, quant=F8)
    assert y.shape == (0, 256) and q.shape == (0, 256) and scale.shape == (0, 2)
    x = torch.randint(0, 9, ((1 << 21) + 3, 8), device="cuda", dtype=torch.int32).to(BF16)  # more workgroups than one grid dimension takes
    got = moe.moe_rmsnorm_add(x, w[:8], 1e-6)[1]
    y = _reference(x, None, w[:8], 1e-6, NONE)[1]
    ru.assert_close(got, y, 4.6 * U * y.abs())


def test_rows_past_four_gib():
    """More than 2^32 bytes of rows: the last ones are those of a small call."""
    T, H = (1 << 17) + 3, 16384
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    x[-4:] = _rand((4, H), BF16, 4)
    x[0] = x[-1]
    w = _weight(H, BF16, 5)
    _, y, q, scale = moe.moe_rmsnorm_add(x, w, 1e-6, quant=I8)
    few = moe.moe_rmsnorm_add(x[-4:].contiguous(), w, 1e-6, quant=I8)
    assert torch.equal(y[-4:], few[1]) and torch.equal(q[-4:], few[2]) and torch.equal(scale[-4:], few[3])
    assert torch.equal(y[0], y[-1]) and not bool(y[1:-4].any())
    del x, q
    dy = torch.zeros((T, H), dtype=BF16, device="cuda")
    dy[-4:] = few[1]
    dx, dw = moe.moe_rmsnorm_add_grad(dy, y, w, 1e-6)
    small = moe.moe_rmsnorm_add_grad(dy[-4:].contiguous(), y[-4:].contiguous(), w, 1e-6)
    assert torch.equal(dx[-4:], small[0])


def _grad_reference(dy, s, w, eps, ds):
    """(dx, dw) in 64 bits with the bounds of their fp32 arithmetic."""
    v, d, wd = s.double(), dy.double(), w.double()
    H = v.shape[1]
    r = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)
    xhat = v * r
    a, c = r * d * wd, (d * wd * v).mean(dim=1, keepdim=True) * r * r
    add = 0.0 if ds is None else ds.double()
    dx = a - xhat * c + add
    # a: g, r and the product rounded; xhat c: xhat (r and the product), c (its sum's terms d w rounded to fp32, and itself);
    # the difference and the sum with ds rounded
    mass_c = (d * wd * v).abs().mean(dim=1, keepdim=True) * r * r
    err = U * (5 * a.abs() + xhat.abs() * (5 * c.abs() + mass_c) + (add.abs() if ds is not None else 0.0)) * 1.01
    dw = (d * xhat).sum(dim=0)
    return dx, err, dw, (d * xhat).abs().sum(dim=0)


def _check_grad(dy, s, w, eps, ds, got):
    T, H = s.shape
    dx, err, dw, mass = _grad_reference(dy, s, w, eps, ds)
    ru.assert_close(got[0], dx, err, "dx")
    # a workgroup adds at most T / parts rows in fp32 (one rounding each), xhat is off by 2^-23; the parts are added in 64 bits
    parts = max(1, moe.moe_rmsnorm_add_grad_workspace_bytes(T, H) // (4 * H))
    ru.assert_close(got[1], dw, (-(-T // parts) + 3) * U * mass, "dw")


@pytest.mark.parametrize("T,H", [(1, 8), (3, 40), (5, 512), (77, 2048), (2, 1048), (700, 520), (9, 4096), (1100, 264), (3, 8192), (1040, 4096),
                                 (2, 8448), (300, 16384), (5000, 64)])
@pytest.mark.parametrize("x_dtype,w_dtype,out", [(BF16, BF16, None), (BF16, F32, None), (F16, F16, F32), (F16, F32, BF16)])
def test_grad(T, H, x_dtype, w_dtype, out):
    dy, s, ds, w = _rand((T, H), x_dtype, T), _rand((T, H), x_dtype, T + 1, 2.0), _rand((T, H), x_dtype, T + 2), _weight(H, w_dtype, H)
    out_dtype = {None: None, F32: moe.MOE_OUT_F32, BF16: moe.MOE_OUT_BF16}[out]
    for more in (None, ds):
        got = moe.moe_rmsnorm_add_grad(dy, s, w, 1e-5, ds=more, out_dtype=out_dtype)
        assert got[1].dtype == (out or w_dtype)
        _check_grad(dy, s, w, 1e-5, more, got)


def test_grad_against_differences():
    """The formula's gradient is that of the 64-bit norm (central differences: error of h^2 / 6 times the third derivative,
    and 2^-52 / h), and the operator's is the formula's."""
    T, H, eps, h = 3, 64, 1e-5, 1e-5
    s, w, dy = _rand((T, H), F16, 1), _weight(H, F32, 2), _rand((T, H), F16, 3)
    f = lambda v, wd: (v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps) * wd * dy.double()).sum()
    dx, err, dw, mass = _grad_reference(dy, s, w, eps, None)
    for seed in range(4):
        at, along = s.double(), _rand((T, H), F32, 10 + seed).double()
        slope = (f(at + h * along, w.double()) - f(at - h * along, w.double())) / (2 * h)
        assert abs(float(slope - (dx * along).sum())) < 1e-7 * float((dx * along).abs().sum() + 1)
        to = _rand((H,), F32, 20 + seed).double()
        slope = (f(at, w.double() + h * to) - f(at, w.double() - h * to)) / (2 * h)
        assert abs(float(slope - (dw * to).sum())) < 1e-7 * float((dw * to).abs().sum() + 1)
    _check_grad(dy, s, w, eps, None, moe.moe_rmsnorm_add_grad(dy, s, w, eps))


def test_grad_in_place_no_rows_and_same_bits():
    T, H = 900, 1024
    dy, s, ds, w = _rand((T, H), BF16, 1), _rand((T, H), BF16, 2), _rand((T, H), BF16, 3), _weight(H, BF16, 4)
    ref = moe.moe_rmsnorm_add_grad(dy, s, w, 1e-6, ds=ds)
    for name in ("dy", "s", "ds"):
        t = dict(dy=dy.clone(), s=s.clone(), ds=ds.clone())
        ws = torch.full((moe.moe_rmsnorm_add_grad_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
        dx, dw = moe.moe_rmsnorm_add_grad(t["dy"], t["s"], w, 1e-6, ds=t["ds"], dx=t[name], workspace=ws)
        assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    dx, dw = moe.moe_rmsnorm_add_grad(dy[:0], s[:0], w, 1e-6)
    assert dx.shape == (0, H) and not bool(dw.any())
    big = (_rand((2, 256), F32, 6) * 1e30).to(BF16)  # fp32 squares would pass 3.4e38
    _check_grad(_rand((2, 256), BF16, 7), big, w[:256], 1e-6, None, moe.moe_rmsnorm_add_grad(_rand((2, 256), BF16, 7), big, w[:256], 1e-6))


def test_norm_on_a_stream_and_in_a_graph():
    T, H = 33, 2048
    x, r, w = _rand((T, H), BF16, 1), _rand((T, H), BF16, 2), _weight(H, BF16, 3)
    dy = _rand((T, H), BF16, 4)
    ref = moe.moe_rmsnorm_add(x, w, 1e-6, residual=r, quant=F8)
    ref_g = moe.moe_rmsnorm_add_grad(dy, ref[0], w, 1e-6, ds=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_rmsnorm_add(x, w, 1e-6, residual=r, quant=F8, stream=side)
    got_g = moe.moe_rmsnorm_add_grad(dy, got[0], w, 1e-6, ds=r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got + got_g, ref + ref_g):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        out = moe.moe_rmsnorm_add(xs, w, 1e-6, residual=r, quant=F8)
        out_g = moe.moe_rmsnorm_add_grad(dy, out[0], w, 1e-6, ds=r)
    for seed in range(4):
        new = _rand((T, H), BF16, 50 + seed)
        xs.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = moe.moe_rmsnorm_add(new, w, 1e-6, residual=r, quant=F8)
        want_g = moe.moe_rmsnorm_add_grad(dy, want[0], w, 1e-6, ds=r)
        for a, b in zip(out + out_g, want + want_g):
            assert torch.equal(a, b)


def test_two_gradients_of_one_workspace_in_graphs():
    sizes = ((70, 2048), (301, 264))
    ws = torch.full((max(moe.moe_rmsnorm_add_grad_workspace_bytes(*z) for z in sizes),), 0xFF, dtype=torch.uint8, device="cuda")
    args, graphs, outs = [], [], []
    for i, (T, H) in enumerate(sizes):
        args.append((_rand((T, H), BF16, i), _rand((T, H), BF16, 9 + i), _weight(H, F32, 3)))
        _check_grad(*args[-1], 1e-6, None, moe.moe_rmsnorm_add_grad(*args[-1], 1e-6, workspace=ws))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(moe.moe_rmsnorm_add_grad(*args[-1], 1e-6, workspace=ws))
    for seed in range(4):
        for dy, _, _ in args:
            dy.copy_(_rand(tuple(dy.shape), BF16, 70 + seed))
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for a, out in zip(args, outs):
            want = moe.moe_rmsnorm_add_grad(*a, 1e-6)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_codes_feed_the_products():
    """norm -> int8 codes -> moe_gemm_i8, and norm -> products by expert -> their gradients -> the norm's gradient."""
    T, H, N, E = 24, 512, 96, 3
    x, r, w = _rand((T, H), BF16, 1), _rand((T, H), BF16, 2), _weight(H, BF16, 3)
    s, y, q, scale = moe.moe_rmsnorm_add(x, w, 1e-6, residual=r, quant=I8)
    Wq, Ws = moe.moe_i8_quantize(_rand((N, H), F32, 4, H ** -0.5))
    C = moe.moe_gemm_i8(q, scale, Wq, Ws, out_dtype=moe.MOE_OUT_F32)
    ref = (q.double() * scale.double()[:, None]) @ (Wq.double() * Ws.double()[:, None]).t()
    ru.assert_close(C, ref, 4 * U * ref.abs())  # exact sums, the scales' product and its product with the sum rounded
    counts = [10, 0, 14]
    W = _rand((E, N, H), BF16, 5, H ** -0.5)
    off = ru.offsets_of(counts)
    out = moe.moe_grouped_gemm_w16(y, None, 1, W, off, T)
    C, mass = ru.grouped(y, W, counts)
    ru.assert_close(out, C, ru.sum_bound(H, mass))
    dC = _rand((T, N), BF16, 6)
    dy = moe.moe_grouped_gemm_w16_dx(dC, W, off)
    _check_grad(dy, s, w, 1e-6, r, moe.moe_rmsnorm_add_grad(dy, s, w, 1e-6, ds=r))


def test_refusals_of_the_binding():
    x, w = _rand((4, 128), BF16, 1), _weight(128, BF16, 2)
    bad = [lambda: moe.moe_rmsnorm_add(x.float(), w, 1e-6), lambda: moe.moe_rmsnorm_add(x, w.half(), 1e-6),
           lambda: moe.moe_rmsnorm_add(x, w[:64], 1e-6), lambda: moe.moe_rmsnorm_add(x, w, 1e-6, residual=x[:2]),
           lambda: moe.moe_rmsnorm_add(x.t(), w, 1e-6), lambda: moe.moe_rmsnorm_add(x, w, 1e-6, s=x),
           lambda: moe.moe_rmsnorm_add(x, w, 1e-6, quant=9), lambda: moe.moe_rmsnorm_add(x, w, 1e-6, q=x),
           lambda: moe.moe_rmsnorm_add(x[:, :64].contiguous(), w[:64], 1e-6, quant=F8),
           lambda: moe.moe_rmsnorm_add(x, w, 1e-6, quant=I8, q=torch.zeros((4, 128), dtype=torch.uint8, device="cuda")),
           lambda: moe.moe_rmsnorm_add_grad(x, x, w, 1e-6, ds=x.half()), lambda: moe.moe_rmsnorm_add_grad(x[:2], x, w, 1e-6),
           lambda: moe.moe_rmsnorm_add_grad(x, x, w, 1e-6, out_dtype=77)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoEError):
        moe.moe_rmsnorm_add(x, w, 0.0)
    with pytest.raises(moe.MoEError):
        moe.moe_rmsnorm_add(x, w, 1e-6, want_y=False)
    with pytest.raises(moe.MoEError):
        moe.moe_rmsnorm_add_grad(x, x, w, 1e-6, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("x_dtype,w_dtype", [(BF16, BF16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("T,H", [(7, 512), (2050, 1024), (33, 2048), (6, 16384)])
def test_y_does_not_depend_on_the_codes(T, H, x_dtype, w_dtype):
    """The same bits of y whatever codes are formed beside it, in rows of ordinary and of far magnitudes, of products past fp32
    and (every 16th column, where y itself is ordinary) below its normal range."""
    x, w = _rand((T, H), F32, T), _weight(H, F32, H)
    eps = 1e-6
    if x_dtype == BF16:
        eps = 2.0 ** -100
        x[1] *= 1e30
        x[2] *= 1e-36
        x[3] *= 2.0 ** -38
        x[3, 5::16] *= 2.0 ** -52
        x[4] *= 2.0 ** 100
        x[5] *= 2.0 ** 50
        w[5::16] *= 2.0 ** -57
        w[9] *= 2.0 ** 75
    x, w = x.to(x_dtype), w.to(w_dtype)
    plain = moe.moe_rmsnorm_add(x, w, eps)
    _check(x, None, w, eps, NONE, True, plain)
    for quant in (I8, F8):
        got = moe.moe_rmsnorm_add(x, w, eps, quant=quant)
        assert torch.equal(got[1], plain[1])
        _check(x, None, w, eps, quant, True, got)


def test_weight_gradient_of_many_rows():
    """However many rows there are, at most 256 of them are added one after the other in fp32 (and then 3 waves' sums); the rest is
    added in 64 bits.  Every addend is 1/2 + 2^-14 - 2^-21, which a sum of 2048 such rows on rounds down by almost half a step each time."""
    T, H = 1 << 24, 8
    r = 1 + 2.0 ** -13 - 2.0 ** -20
    eps = float(torch.tensor(1 / r ** 2 - 0.25, dtype=F32))
    s, dy = torch.full((T, H), 0.5, dtype=BF16, device="cuda"), torch.ones((T, H), dtype=BF16, device="cuda")
    _, dw = moe.moe_rmsnorm_add_grad(dy, s, torch.ones(H, device="cuda"), eps)
    want = torch.full((H,), T * 0.5 / (0.25 + eps) ** 0.5, dtype=torch.float64, device="cuda")
    ru.assert_close(dw, want, (256 + 6) * U * want, "dw")
