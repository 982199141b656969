"""The ragged products (int8 and 16-bit weights), their gradients, and SiLU*mul, against plain forms in 64
bits, at the sizes and group shapes where they can go wrong."""
from fractions import Fraction

import pytest
import torch

import moe_w4a16_grouped_amd as moe
from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
OUT = {BF16: moe.MOE_OUT_BF16, F16: moe.MOE_OUT_F16, F32: moe.MOE_OUT_F32}
SILU, NONE = moe.MOE_EPI_SILU_MUL, moe.MOE_EPI_NONE

# counts of the groups: mean rows in each range of the tile choice, empty groups in front, between and behind,
# one row, groups one past and one short of a tile, a single group
GROUPS = {
    "one_row": [0, 1, 0],
    "decode": [0, 3, 1, 0, 0, 16, 17, 2],
    "mean24": [33, 0, 15, 48],
    "mean50": [64, 65, 0, 70],
    "mean200": [0, 128, 129, 500, 43],
    "mean400": [257, 0, 1100, 243],
    "single": [300],
}


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _case(counts, T, K, dtype, seed):
    """Tokens [T, K] and a gather of sum(counts) rows from them (flat index / 3), with repeats."""
    R = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = _rand((T, K), dtype, seed + 1)
    row_of = torch.randint(0, 3 * T, (R,), generator=g, device="cuda", dtype=torch.int32)
    return x, row_of, x[(row_of // 3).long()]


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K,dtype,out,epi", [
    (256, 256, BF16, BF16, NONE), (130, 72, F16, F32, NONE), (7, 8, BF16, F32, NONE), (514, 328, BF16, BF16, SILU),
    (6, 1000, F16, F16, SILU), (1, 136, F16, F16, NONE)])
def test_grouped_w16(name, N, K, dtype, out, epi):
    counts = GROUPS[name]
    x, row_of, rows = _case(counts, 40, K, dtype, seed=N + K)
    W = _rand((len(counts), N, K), dtype, 7, K ** -0.5)
    C = moe.moe_grouped_gemm_w16(x, row_of, 3, W, ru.offsets_of(counts), sum(counts), epilogue=epi, out_dtype=OUT[out])
    ref, mass = ru.grouped(rows, W, counts)
    err = ru.sum_bound(K, mass)
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(C, ref, err, f"{name} {N} {K}")


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K,dtype,out", [(256, 256, BF16, BF16), (72, 136, F16, F32), (8, 8, BF16, F32), (328, 520, F16, F16)])
def test_grouped_w16_gradients(name, N, K, dtype, out):
    counts = GROUPS[name]
    R = sum(counts)
    x, row_of, rows = _case(counts, 50, K, dtype, seed=N + K)
    W, dC = _rand((len(counts), N, K), dtype, 3, K ** -0.5), _rand((R, N), dtype, 4)
    off = ru.offsets_of(counts)
    dA = moe.moe_grouped_gemm_w16_dx(dC, W, off, out_dtype=OUT[out])
    ref, mass = ru.grouped(dC, W.transpose(1, 2), counts)
    ru.assert_close(dA, ref, ru.sum_bound(N, mass), f"dA {name}")
    dW = torch.full((len(counts), N, K), float("nan"), dtype=out, device="cuda")
    moe.moe_grouped_gemm_w16_dw(dC, x, row_of, 3, off, out_dtype=OUT[out], dW=dW)
    ref, mass = ru.grouped_dw(dC, rows, counts)
    ru.assert_close(dW, ref, ru.sum_bound(max(counts), mass), f"dW {name}")
    dW2 = moe.moe_grouped_gemm_w16_dw(dC, rows.contiguous(), None, 1, off, out_dtype=OUT[out])
    assert torch.equal(dW, dW2)


@pytest.mark.parametrize("counts", [[0, 2500, 100, 3], [0, 9001, 5, 100]])
def test_weight_gradients_of_long_groups(counts):
    """Groups longer than the gathered indexes kept at a time, in both tile choices."""
    N, K, R = 136, 264, sum(counts)
    if counts[1] == 2500:
        counts = counts + [0] * 12  # mean rows of the small tile choice
    x, row_of, rows = _case(counts, 700, K, BF16, seed=5)
    dC = _rand((R, N), BF16, 6)
    dW = moe.moe_grouped_gemm_w16_dw(dC, x, row_of, 3, ru.offsets_of(counts), out_dtype=moe.MOE_OUT_F32)
    ref, mass = ru.grouped_dw(dC, rows, counts)
    ru.assert_close(dW, ref, ru.sum_bound(max(counts), mass))


@pytest.mark.parametrize("counts,N,K,out", [([4000], 128, 256, F16), ([700, 0, 33, 5000], 72, 104, F32),
                                            ([31, 2049], 264, 8, BF16)])
def test_weight_gradients_in_parts(counts, N, K, out):
    """Few weights with many rows: the rows are cut into parts; groups shorter than a part, empty ones, ends inside
    one, gathered and plain rows, and the parts' sums added the same way each time."""
    R, E = sum(counts), len(counts)
    assert moe.moe_grouped_gemm_w16_dw_workspace_bytes(R, E, N, K) > 0
    x, row_of, rows = _case(counts, 500, K, BF16, seed=9)
    dC, off = _rand((R, N), BF16, 10), ru.offsets_of(counts)
    dW = moe.moe_grouped_gemm_w16_dw(dC, x, row_of, 3, off, out_dtype=OUT[out])
    ref, mass = ru.grouped_dw(dC, rows, counts)
    ru.assert_close(dW, ref, ru.sum_bound(max(counts), mass))
    assert torch.equal(dW, moe.moe_grouped_gemm_w16_dw(dC, rows.contiguous(), None, 1, off, out_dtype=OUT[out]))


# calls that fill the card, one for each range of the tile choice: (experts, counts drawn from)
FULL = {
    "decode": (200, [0, 0, 1, 2, 16, 17]),
    "mean20": (200, [0, 1, 15, 16, 17, 31, 32, 33, 50]),
    "mean50": (120, [0, 1, 33, 63, 64, 65, 129]),
    "mean200": (100, [0, 1, 127, 128, 129, 255, 256, 257, 500]),
    "mean600": (50, [0, 1, 128, 129, 256, 385, 512, 1100, 2000]),
}


def _full(name):
    E, pick = FULL[name]
    g = torch.Generator().manual_seed(E)
    return [pick[i] for i in torch.randint(0, len(pick), (E,), generator=g).tolist()]


@pytest.mark.parametrize("name", list(FULL))
@pytest.mark.parametrize("N,K,dtype,out,epi", [(520, 264, BF16, BF16, NONE), (514, 136, F16, F32, NONE), (516, 72, F16, F32, NONE),
                                               (514, 40, BF16, F16, NONE), (1040, 520, BF16, BF16, SILU), (1030, 8, F16, F16, SILU)])
def test_full_grid_w16(name, N, K, dtype, out, epi):
    counts = _full(name)
    x, row_of, rows = _case(counts, 333, K, dtype, seed=N + K)
    W = _rand((len(counts), N, K), dtype, 7, K ** -0.5)
    C = moe.moe_grouped_gemm_w16(x, row_of, 3, W, ru.offsets_of(counts), sum(counts), epilogue=epi, out_dtype=OUT[out])
    ref, mass = ru.grouped(rows, W, counts)
    err = ru.sum_bound(K, mass)
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(C, ref, err, f"{name} {N} {K}")


@pytest.mark.parametrize("counts", [[700, 0, 580], [1280], [256, 256, 300, 129, 257], [1, 1400]])
@pytest.mark.parametrize("dtype,out,epi", [(BF16, BF16, NONE), (F16, F32, NONE), (BF16, BF16, SILU)])
def test_last_round_in_halves(counts, dtype, out, epi):
    """A little more than one round of the highest tiles on the card, whose last ones are cut in halves."""
    N, K, R = 14336, 2056, sum(counts)
    A, W = _rand((R, K), dtype, 1), _rand((len(counts), N, K), dtype, 2, K ** -0.5)
    C = moe.moe_grouped_gemm_w16(A, None, 1, W, ru.offsets_of(counts), R, epilogue=epi, out_dtype=OUT[out])
    ref, mass = ru.grouped(A, W, counts)
    err = ru.sum_bound(K, mass)
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(C, ref, err, counts)
    q, s = moe.moe_i8_quantize(A[:, :2048].contiguous().repeat(1, 2))
    wq, ws = moe.moe_i8_quantize(W[0, :, :2048].repeat(1, 2))
    C = moe.moe_gemm_i8(q, s, wq, ws, epilogue=epi, out_dtype=OUT[out])
    ref, err = _i8_reference(q, s, wq, ws)
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(C, ref, err, counts)


@pytest.mark.parametrize("name", list(FULL))
@pytest.mark.parametrize("N,K,dtype,out", [(520, 520, BF16, BF16), (264, 1032, F16, F32), (776, 392, F16, F16)])
def test_full_grid_w16_gradients(name, N, K, dtype, out):
    counts = _full(name)
    R = sum(counts)
    x, row_of, rows = _case(counts, 333, K, dtype, seed=N + K)
    W, dC = _rand((len(counts), N, K), dtype, 3, K ** -0.5), _rand((R, N), dtype, 4)
    off = ru.offsets_of(counts)
    dA = moe.moe_grouped_gemm_w16_dx(dC, W, off, out_dtype=OUT[out])
    ref, mass = ru.grouped(dC, W.transpose(1, 2), counts)
    ru.assert_close(dA, ref, ru.sum_bound(N, mass), f"dA {name}")
    dW = moe.moe_grouped_gemm_w16_dw(dC, x, row_of, 3, off, out_dtype=OUT[out])
    ref, mass = ru.grouped_dw(dC, rows, counts)
    ru.assert_close(dW, ref, ru.sum_bound(max(counts), mass), f"dW {name}")
    assert torch.equal(dW, moe.moe_grouped_gemm_w16_dw(dC, rows.contiguous(), None, 1, off, out_dtype=OUT[out]))


def test_gradients_against_differences():
    """dA and dW against central differences of the 64-bit product along random directions: the loss
    sum(C * dC) is linear in A and in W, so a difference quotient is exact up to rounding."""
    counts, N, K = [5, 0, 40, 3], 48, 64
    off, R = ru.offsets_of(counts), 48
    A, W, dC = _rand((R, K), BF16, 1), _rand((4, N, K), BF16, 2), _rand((R, N), BF16, 3)
    dA = moe.moe_grouped_gemm_w16_dx(dC, W, off, out_dtype=moe.MOE_OUT_F32).double()
    dW = moe.moe_grouped_gemm_w16_dw(dC, A, None, 1, off, out_dtype=moe.MOE_OUT_F32).double()
    loss = lambda a, w: float((ru.grouped(a, w, counts)[0] * dC.double()).sum())
    da, dw = _rand((R, K), F32, 4).double(), _rand((4, N, K), F32, 5).double()
    errs = ru.sum_bound(N, ru.grouped(dC, W.transpose(1, 2), counts)[1]), ru.sum_bound(40, ru.grouped_dw(dC, A, counts)[1])
    for grad, err, step, plus, minus in ((dA, errs[0], da, (A.double() + da, W.double()), (A.double() - da, W.double())),
                                         (dW, errs[1], dw, (A.double(), W.double() + dw), (A.double(), W.double() - dw))):
        num, ana = (loss(*plus) - loss(*minus)) / 2, float((grad * step).sum())
        assert abs(num - ana) <= float(((err + 2.0 ** -24 * grad.abs()) * step.abs()).sum())


def test_rows_past_the_groups_are_left_alone():
    counts, R = [3, 0, 20], 40
    off = ru.offsets_of(counts)
    A, W = _rand((R, 64), BF16, 1), _rand((3, 32, 64), BF16, 2)
    C = torch.full((R, 32), 5.0, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_w16(A, None, 1, W, off, R, C=C)
    assert torch.all(C[23:] == 5.0)
    ref, mass = ru.grouped(A[:23], W, counts)
    ru.assert_close(C[:23], ref, ru.sum_bound(64, mass))
    dA = torch.full((R, 64), 5.0, dtype=BF16, device="cuda")
    dC = _rand((R, 32), BF16, 3)
    moe.moe_grouped_gemm_w16_dx(dC, W, off, dA=dA)
    assert torch.all(dA[23:] == 5.0)
    q, s = moe.moe_i8_quantize(A)
    wq, ws = moe.moe_i8_quantize(W.view(-1, 64))
    C = torch.full((R, 32), 5.0, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_i8(q, s, None, 1, wq.view(3, 32, 64), ws.view(3, 32), off, R, C=C)
    assert torch.all(C[23:] == 5.0)
    # rows behind the groups add nothing to the weight gradients
    dW = moe.moe_grouped_gemm_w16_dw(dC, A, None, 1, off)
    dW2 = moe.moe_grouped_gemm_w16_dw(dC[:23].contiguous(), A, None, 1, off)
    assert torch.equal(dW, dW2)


def test_offsets_are_clamped_to_the_rows():
    """Offsets past the rows end at them."""
    R = 30
    A, W, dC = _rand((R, 64), BF16, 1), _rand((2, 32, 64), BF16, 2), _rand((R, 32), BF16, 3)
    off = torch.tensor([0, 10, 1000], dtype=torch.int32, device="cuda")
    ok = ru.offsets_of([10, 20])
    assert torch.equal(moe.moe_grouped_gemm_w16(A, None, 1, W, off, R), moe.moe_grouped_gemm_w16(A, None, 1, W, ok, R))
    assert torch.equal(moe.moe_grouped_gemm_w16_dx(dC, W, off), moe.moe_grouped_gemm_w16_dx(dC, W, ok))
    assert torch.equal(moe.moe_grouped_gemm_w16_dw(dC, A, None, 1, off), moe.moe_grouped_gemm_w16_dw(dC, A, None, 1, ok))


def test_no_rows():
    W, off = _rand((3, 32, 64), BF16, 1), ru.offsets_of([0, 0, 0])
    empty = torch.empty((0, 64), dtype=BF16, device="cuda")
    assert moe.moe_grouped_gemm_w16(empty, None, 1, W, off, 0).shape == (0, 32)
    assert moe.moe_grouped_gemm_w16_dx(torch.empty((0, 32), dtype=BF16, device="cuda"), W, off).shape == (0, 64)
    dW = torch.full((3, 32, 64), float("nan"), dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_w16_dw(torch.empty((0, 32), dtype=BF16, device="cuda"), empty, None, 1, off, dW=dW)
    assert torch.all(dW == 0)
    q, s = moe.moe_i8_quantize(empty)
    assert q.shape == (0, 64) and s.shape == (0,)
    wq, ws = moe.moe_i8_quantize(W[0].contiguous())
    assert moe.moe_linear_i8(empty, wq, ws).shape == (0, 32)
    assert moe.moe_silu_mul(empty).shape == (0, 32)


def test_non_finite_rows_stay_in_their_rows():
    counts = [20, 0, 300, 5]
    R, N, K = 325, 72, 104
    off = ru.offsets_of(counts)
    A, W, dC = _rand((R, K), BF16, 1), _rand((4, N, K), BF16, 2), _rand((R, N), BF16, 3)
    bad = [19, 20, 319]
    A2, dC2 = A.clone(), dC.clone()
    A2[bad, 5], dC2[bad, 6] = float("nan"), float("inf")
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[bad] = False
    C, C2 = (moe.moe_grouped_gemm_w16(a, None, 1, W, off, R) for a in (A, A2))
    assert torch.equal(C[keep], C2[keep]) and not torch.isfinite(C2[bad]).any()
    D, D2 = (moe.moe_grouped_gemm_w16_dx(d, W, off) for d in (dC, dC2))
    assert torch.equal(D[keep], D2[keep]) and not torch.isfinite(D2[bad]).any()
    G, G2 = (moe.moe_grouped_gemm_w16_dw(d, a, None, 1, off) for d, a in ((dC, A), (dC2, A2)))
    assert torch.equal(G[3], G2[3]) and torch.equal(G[1], G2[1])
    assert torch.equal(G[0][7:, 6:], G2[0][7:, 6:]) and not torch.isfinite(G2[0][6]).any()
    A2, W, K = A2[:, :96].contiguous(), W[:, :, :96].contiguous(), 96  # int8 rows are whole 16-byte chunks
    q, s = moe.moe_i8_quantize(A2)
    assert torch.isnan(s[bad]).all() and (q[bad] == 0).all() and torch.isfinite(s[keep]).all()
    wq, ws = moe.moe_i8_quantize(W.view(-1, K))
    Y = moe.moe_grouped_gemm_i8(q, s, None, 1, wq.view(4, N, K), ws.view(4, N), off, R)
    assert torch.isnan(Y[bad]).all() and torch.isfinite(Y[keep]).all()


# ---- int8 --------------------------------------------------------------------------------------------

def _codes_64(x):
    """Codes and scales by the definition, the quotient in 64 bits (bf16 / fp16 x: 11 bits over 24, so the
    64-bit quotient tells every real quotient from a half)."""
    x = x.double()
    s = (x.abs().amax(dim=1) / 127).float()
    q = torch.round(x / torch.where(s > 0, s, 1).double()[:, None])
    return torch.where(s[:, None] > 0, q, 0).to(torch.int8), s


@pytest.mark.parametrize("rows,K,dtype", [(1, 16, BF16), (7, 528, BF16), (300, 2048, F16), (33, 4112, F32), (5, 8208, BF16),
                                          (2, 16384, F16), (64, 512, F32)])
def test_i8_quantize(rows, K, dtype):
    x = _rand((rows, K), dtype, rows + K)
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-3
    q, s = moe.moe_i8_quantize(x)
    rq, rs = _codes_64(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)


def test_i8_quantize_ties_and_neighbours():
    """Quotients on a half, and one fp32 step to either side: the codes are those of the exact quotient."""
    s = torch.tensor([1.0, 0.37109375, 3.0], dtype=torch.float64)
    n = torch.arange(-126, 126, dtype=torch.float64) + 0.5
    rows = []
    for v in s:
        mid = (n * v).float()  # exact: n has 8 bits, v at most 7
        rows += [mid, torch.nextafter(mid, torch.tensor(1e9)), torch.nextafter(mid, torch.tensor(-1e9))]
    x = torch.stack(rows)
    top = (127 * s).float().repeat_interleave(3)[:, None].expand(-1, 4)
    x = torch.cat([x, top], dim=1)  # the largest magnitude makes the scale v
    want = torch.empty_like(x)
    for i in range(x.shape[0]):
        v = float(s[i // 3])
        for j in range(x.shape[1]):
            want[i, j] = round(Fraction(float(x[i, j])) / Fraction(v))  # round: ties to even
    q, sc = moe.moe_i8_quantize(x.cuda())
    assert torch.equal(sc.cpu().double(), s.repeat_interleave(3))
    assert torch.equal(q.cpu().float(), want)


def test_i8_quantize_extremes():
    x = torch.zeros((4, 32), dtype=F32)
    x[0, 3] = 3e38
    x[1, 4] = 1e-44   # its scale rounds to 0: codes 0
    x[2, 5] = -1e-38
    x[3, :] = -2.0
    q, s = moe.moe_i8_quantize(x.cuda())
    q, s = q.cpu(), s.cpu()
    assert q[0, 3] == 127 and q[0].count_nonzero() == 1
    assert s[1] == 0 and not q[1].any()
    assert q[2, 5] == -127
    assert torch.all(q[3] == -127)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -70, 2.0 ** -110, 2.0 ** -126])
def test_i8_quantize_tiny_rows(scale):
    """Rows whose scale is near the least fp32 number or subnormal, zeros among them, in every path of the codes."""
    for rows, K, dtype in ((3, 64, F32), (40, 1040, BF16), (2, 8208, F32)):
        x = (_rand((rows, K), F32, K) * scale).to(dtype)
        x[:, ::5] = 0
        q, s = moe.moe_i8_quantize(x)
        rq, rs = _codes_64(x)
        rq = torch.where(rs[:, None] > 0, torch.round(x.double() / rs.double()[:, None]).clamp(-127, 127), 0).to(torch.int8)
        assert torch.equal(s, rs) and torch.equal(q, rq), (rows, K)
        if dtype == F32:
            w = torch.ones((8, K), dtype=torch.int8, device="cuda")
            y = moe.moe_linear_i8(x, w, torch.full((8,), 2.0 ** 60, device="cuda"), out_dtype=OUT[F32])
            ref, err = _i8_reference(q, s, w, torch.full((8,), 2.0 ** 60, device="cuda"))
            ru.assert_close(y, ref, err, (rows, K))


def test_i8_quantize_many_rows():
    """The most rows: more threads than a launch dimension holds."""
    rows = 2 ** 26 - 1
    x = torch.zeros((rows, 16), dtype=BF16, device="cuda")
    at = torch.tensor([0, 2 ** 19 - 1, 2 ** 19, 2 ** 24 - 1, 2 ** 24, 2 ** 25 + 3, rows - 1], device="cuda")
    x[at] = _rand((at.numel(), 16), BF16, 7)
    q, s = moe.moe_i8_quantize(x)
    rq, rs = _codes_64(x[at])
    assert torch.equal(s[at], rs) and torch.equal(q[at], rq)
    assert int((s != 0).sum()) == at.numel() and int(q.view(torch.int32).ne(0).any(dim=1).sum()) == at.numel()


def _i8_reference(q, s, wq, ws):
    """(G, error): the integer sums are exact; the sum's conversion, the scales' product and their product round
    once each."""
    G = (q.double() @ wq.double().t()) * (s.double()[:, None] * ws.double())
    return G, 3.01 * 2.0 ** -24 * G.abs()


@pytest.mark.parametrize("T", [1, 5, 16, 17, 50, 130, 300])
@pytest.mark.parametrize("N,K,dtype,out,epi", [(256, 256, BF16, BF16, NONE), (131, 144, F16, F32, NONE), (258, 2064, F32, F16, SILU),
                                               (2, 16, BF16, BF16, SILU), (1, 48, F16, F16, NONE)])
def test_linear_i8(T, N, K, dtype, out, epi):
    x, w = _rand((T, K), dtype, T), _rand((N, K), F32, N, K ** -0.5)
    wq, ws = moe.moe_i8_quantize(w)
    y = moe.moe_linear_i8(x, wq, ws, epilogue=epi, out_dtype=OUT[out])
    q, s = _codes_64(x)
    ref, err = _i8_reference(q, s, wq, ws)
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(y, ref, err)
    q2, s2 = moe.moe_i8_quantize(x)
    assert torch.equal(y, moe.moe_gemm_i8(q2, s2, wq, ws, epilogue=epi, out_dtype=OUT[out]))


@pytest.mark.parametrize("T,K", [(1, 16), (1, 8192), (2, 4096), (3, 2720), (4, 2048), (5, 1632), (8, 1024), (9, 896), (12, 672), (16, 512), (16, 16)])
@pytest.mark.parametrize("N,dtype,out,epi", [(70, BF16, BF16, NONE), (4200, F16, F32, NONE), (100, F32, F16, SILU), (38, BF16, BF16, SILU)])
def test_linear_i8_of_few_rows(T, K, N, dtype, out, epi):
    """The most that one launch takes of each number of rows, with columns that end inside a block."""
    x, (wq, ws) = _rand((T, K), dtype, T), moe.moe_i8_quantize(_rand((N, K), F32, N, K ** -0.5))
    y = moe.moe_linear_i8(x, wq, ws, epilogue=epi, out_dtype=OUT[out])
    q, s = moe.moe_i8_quantize(x)
    ref, err = _i8_reference(q, s, wq, ws)
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(y, ref, err)
    assert torch.equal(y, moe.moe_gemm_i8(q, s, wq, ws, epilogue=epi, out_dtype=OUT[out]))


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K,out,epi", [(256, 256, BF16, SILU), (133, 80, F32, NONE), (260, 1040, F16, NONE)])
def test_grouped_i8(name, N, K, out, epi):
    counts = GROUPS[name]
    E, R = len(counts), sum(counts)
    x, row_of, rows = _case(counts, 60, K, BF16, seed=K)
    wq, ws = moe.moe_i8_quantize(_rand((E * N, K), F32, 2, K ** -0.5))
    wq, ws = wq.view(E, N, K), ws.view(E, N)
    q, s = moe.moe_i8_quantize(x)
    C = moe.moe_grouped_gemm_i8(q, s, row_of, 3, wq, ws, ru.offsets_of(counts), R, epilogue=epi, out_dtype=OUT[out])
    at, parts = 0, []
    tok = (row_of // 3).long()
    for e, n in enumerate(counts):
        parts.append(_i8_reference(q[tok[at:at + n]], s[tok[at:at + n]], wq[e], ws[e]))
        at += n
    ref, err = (torch.cat(p) for p in zip(*parts))
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(C, ref, err, name)


@pytest.mark.parametrize("name", list(FULL))
@pytest.mark.parametrize("N,K,out,epi", [(520, 272, BF16, NONE), (514, 144, F32, NONE), (516, 528, F32, NONE), (1040, 400, F16, SILU)])
def test_full_grid_i8(name, N, K, out, epi):
    counts = _full(name)
    E, R = len(counts), sum(counts)
    x, row_of, _ = _case(counts, 333, K, BF16, seed=K)
    wq, ws = moe.moe_i8_quantize(_rand((E * N, K), F32, 2, K ** -0.5))
    q, s = moe.moe_i8_quantize(x)
    C = moe.moe_grouped_gemm_i8(q, s, row_of, 3, wq.view(E, N, K), ws.view(E, N), ru.offsets_of(counts), R, epilogue=epi, out_dtype=OUT[out])
    tok = (row_of // 3).long()
    e_of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    exact, _ = ru.grouped(q[tok].float(), wq.view(E, N, K).float(), counts)
    ref = exact * (s.double()[tok, None] * ws.view(E, N).double()[e_of])
    err = 3.01 * 2.0 ** -24 * ref.abs()  # as in _i8_reference
    if epi == SILU:
        ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(C, ref, err, name)


@pytest.mark.parametrize("M", [900, 4097])
def test_dense_i8_of_many_columns(M):
    """One group with enough columns for the large tiles."""
    N, K = 12808, 80
    q, s = moe.moe_i8_quantize(_rand((M, K), BF16, 1))
    wq, ws = moe.moe_i8_quantize(_rand((N, K), F32, 2, K ** -0.5))
    ref, err = _i8_reference(q, s, wq, ws)
    ru.assert_close(moe.moe_gemm_i8(q, s, wq, ws), ref, err)
    ref, err = ru.silu_mul(ref), ru.silu_bound(ref, err)
    ru.assert_close(moe.moe_gemm_i8(q, s, wq, ws, epilogue=SILU), ref, err)


def test_i8_sums_stay_exact_at_the_largest_K():
    K = 1 << 17
    q = torch.full((3, K), 127, dtype=torch.int8, device="cuda")
    q[1] = -127
    q[2, ::2] = -127
    one = torch.ones(3, device="cuda")
    C = moe.moe_gemm_i8(q, one, q, one, out_dtype=moe.MOE_OUT_F32)
    ref = q.double() @ q.double().t()
    assert torch.equal(C.double(), ref.float().double())


# ---- SiLU*mul ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R,I", [(1, 8), (3, 24), (65, 1000), (700, 768)])
def test_silu_mul(R, I, dtype):
    G, dh = _rand((R, 2 * I), dtype, R, 3.0), _rand((R, I), dtype, I)
    G[0, 0], G[0, 1] = 80.0, -80.0
    g, u = G.double().chunk(2, dim=1)
    d, s = dh.double(), torch.sigmoid(g)
    exp_err = 2.0 ** -18 + g.abs() * 2.0 ** -23  # fast exponential and quotient, argument rounding
    ru.assert_close(moe.moe_silu_mul(G), g * s * u, exp_err * (g * s * u).abs())
    dG = moe.moe_silu_mul_grad(G, dh)
    # dg = d u s (1 + g (1 - s)): the error of s enters both factors, 1 - s is off by s's error and a rounding
    es = exp_err * s + 2.0 ** -24
    ref = torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], dim=1)
    err = torch.cat([(d * u).abs() * (exp_err * s * (1 + g * (1 - s)).abs() + s * (g.abs() * es + 2.0 ** -22 * (1 + g.abs()))),
                     exp_err * (d * g * s).abs()], dim=1)
    ru.assert_close(dG, ref, err)
    G2 = G.clone()
    assert torch.equal(moe.moe_silu_mul_grad(G2, dh, dG=G2), dG)  # in place


def test_silu_gradient_against_differences():
    G, dh = _rand((4, 32), BF16, 1), _rand((4, 16), BF16, 2)
    dG = moe.moe_silu_mul_grad(G, dh).double()
    step = 2.0 ** -12
    loss = lambda z: (ru.silu_mul(z) * dh.double()).sum()
    for i, j in ((0, 0), (1, 5), (2, 15), (3, 16), (0, 31)):
        z = torch.zeros((4, 32), dtype=torch.float64, device="cuda")
        z[i, j] = step
        num = float(loss(G.double() + z) - loss(G.double() - z)) / (2 * step)
        # a stored gradient's half step, the third derivative's term (|f'''| < 2, |dh u| < 20) and the fast exponential
        assert abs(num - float(dG[i, j])) <= (2.0 ** -8 + 2.0 ** -17) * abs(num) + 40 * step * step + 2.0 ** -16


# ---- together ----------------------------------------------------------------------------------------

def _route(T, E, k, seed):
    logits = _rand((T, E), F32, seed)
    ids, w = moe.moe_route_topk(logits, k)
    return logits, ids, w, moe.moe_align(ids, E, 64)


def _expert_ffn_64(x, ids, w, w13, w2):
    y = torch.zeros_like(x)
    for s in range(ids.shape[1]):
        for e in ids[:, s].unique():
            t = torch.nonzero(ids[:, s] == e).reshape(-1)
            h = ru.silu_mul(x[t] @ w13[e].t())
            y = y.index_add(0, t, w[t, s, None] * (h @ w2[e].t()))
    return y


def test_training_step_of_the_experts():
    """Forward and backward pass of the expert FFN from the separate operators, against autograd in 64 bits."""
    T, E, k, H, I = 96, 6, 2, 64, 48
    _, ids, w, al = _route(T, E, k, 1)
    off, slots, R = al["offsets"], al["sorted_ids"], T * k
    x, w13, w2 = _rand((T, H), BF16, 2), _rand((E, 2 * I, H), BF16, 3, H ** -0.5), _rand((E, H, I), BF16, 4, I ** -0.5)
    dy = _rand((T, H), BF16, 5)
    G = moe.moe_grouped_gemm_w16(x, slots, k, w13, off, R)
    h = moe.moe_silu_mul(G)
    O = moe.moe_grouped_gemm_w16(h, None, 1, w2, off, R, out_dtype=moe.MOE_OUT_F32)
    y = moe.moe_combine(O, al["inv_perm"], w)
    wr = w.reshape(-1)[slots.long()]
    dO = (dy[(slots // k).long()].float() * wr[:, None]).to(BF16)
    dw2 = moe.moe_grouped_gemm_w16_dw(dO, h, None, 1, off, out_dtype=moe.MOE_OUT_F32)
    dh = moe.moe_grouped_gemm_w16_dx(dO, w2, off)
    dG = moe.moe_silu_mul_grad(G, dh)
    dw13 = moe.moe_grouped_gemm_w16_dw(dG, x, slots, k, off, out_dtype=moe.MOE_OUT_F32)
    dxr = moe.moe_grouped_gemm_w16_dx(dG, w13, off, out_dtype=moe.MOE_OUT_F32)
    dx = moe.moe_combine(dxr, al["inv_perm"], torch.ones_like(w))
    leaves = [t.double().requires_grad_() for t in (x, w13, w2)]
    ref = _expert_ffn_64(leaves[0], ids.long(), w.double(), leaves[1], leaves[2])
    ref.backward(dy.double())
    for name, got, want in (("y", y, ref.detach()), ("dx", dx, leaves[0].grad), ("dw13", dw13, leaves[1].grad),
                            ("dw2", dw2, leaves[2].grad)):
        # four bf16 stores at most on the way (G, h, dO, dh, dG): each adds at most 2^-8 of relative error to
        # what it stores, in the mean of a sum of many such terms
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 5 * 2.0 ** -8, (name, rel)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 64, 48), (9, 16, 4, 128, 80), (150, 8, 3, 272, 144), (1500, 4, 2, 256, 160)])
@pytest.mark.parametrize("kind", ["i8", "w16"])
def test_layers(kind, T, E, k, H, I):
    """The layers equal their steps through the separate entry points, bit for bit."""
    logits, ids, w, al = _route(T, E, k, T)
    x = _rand((T, H), BF16, 2)
    w13, w2 = _rand((E, 2 * I, H), BF16, 3, H ** -0.5), _rand((E, H, I), BF16, 4, I ** -0.5)
    off, slots, R = al["offsets"], al["sorted_ids"], T * k
    ids_out, w_out = torch.empty_like(ids), torch.empty_like(w)
    if kind == "i8":
        w13q, w13s = moe.moe_i8_quantize(w13.view(-1, H))
        w2q, w2s = moe.moe_i8_quantize(w2.view(-1, I))
        w13q, w13s, w2q, w2s = w13q.view(E, 2 * I, H), w13s.view(E, -1), w2q.view(E, H, I), w2s.view(E, -1)
        y = moe.moe_ffn_forward_i8(x, logits, w13q, w13s, w2q, w2s, k, topk_ids_out=ids_out, topk_w_out=w_out)
        q, s = moe.moe_i8_quantize(x)
        h = moe.moe_grouped_gemm_i8(q, s, slots, k, w13q, w13s, off, R, epilogue=SILU)
        q, s = moe.moe_i8_quantize(h)
        O = moe.moe_grouped_gemm_i8(q, s, None, 1, w2q, w2s, off, R, out_dtype=moe.MOE_OUT_F32)
        w13, w2 = w13q.double() * w13s.double()[..., None], w2q.double() * w2s.double()[..., None]
        # 8-bit codes: an error of (largest / rms) / (127 sqrt(12)) of the rms, x 1.0 % (4.5 rms) through gate and up
        # (times 1.6), h 1.8 % (8 rms)
        bound = 3e-2
    else:
        y = moe.moe_ffn_forward_w16(x, logits, w13, w2, k, topk_ids_out=ids_out, topk_w_out=w_out)
        h = moe.moe_grouped_gemm_w16(x, slots, k, w13, off, R, epilogue=SILU)
        O = moe.moe_grouped_gemm_w16(h, None, 1, w2, off, R, out_dtype=moe.MOE_OUT_F32)
        bound = 2 * 2.0 ** -8  # h and y stored in bf16
    assert torch.equal(ids_out, ids) and torch.equal(w_out, w)
    assert torch.equal(y, moe.moe_combine(O, al["inv_perm"], w))
    ref = _expert_ffn_64(x.double(), ids.long(), w.double(), w13.double(), w2.double())
    assert float((y.double() - ref).norm() / ref.norm()) <= bound


# ---- more than 2^32 elements -------------------------------------------------------------------------

def test_results_past_32_bits():
    counts, N, K = [5, 4_200_000, 300], 1040, 16
    R = sum(counts)
    assert R * N > 2 ** 32
    off = ru.offsets_of(counts)
    x, W = _rand((1000, K), BF16, 1), _rand((3, N, K), BF16, 2, K ** -0.5)
    row_of = (torch.arange(R, device="cuda") * 7 % 3000).int()
    C = moe.moe_grouped_gemm_w16(x, row_of, 3, W, off, R)
    h, dA = moe.moe_silu_mul(C), moe.moe_grouped_gemm_w16_dx(C, W, off)
    dG = moe.moe_silu_mul_grad(C, h)
    q, s = moe.moe_i8_quantize(x)
    wq, ws = moe.moe_i8_quantize(W.view(-1, K))
    C8 = moe.moe_grouped_gemm_i8(q, s, row_of, 3, wq.view(3, N, K), ws.view(3, N), off, R)
    edge = 2 ** 32 // N
    for a, b, e in ((0, 5, 0), (5, 70, 1), (edge // 2 - 2, edge // 2 + 2, 1), (edge - 2, edge + 2, 1), (R - 303, R - 300, 1), (R - 300, R, 2)):
        tok = (row_of[a:b] // 3).long()
        ref, mass = ru.grouped(x[tok], W[e:e + 1], [b - a])
        ru.assert_close(C[a:b], ref, ru.sum_bound(K, mass))
        ref, err = _i8_reference(q[tok], s[tok], wq.view(3, N, K)[e], ws.view(3, N)[e])
        ru.assert_close(C8[a:b], ref, err)
        part = C[a:b].contiguous()
        ref, mass = ru.grouped(part, W[e:e + 1].transpose(1, 2), [b - a])
        ru.assert_close(dA[a:b], ref, ru.sum_bound(N, mass))
        assert torch.equal(h[a:b], moe.moe_silu_mul(part)) and torch.equal(dG[a:b], moe.moe_silu_mul_grad(part, h[a:b].contiguous()))


def test_weight_gradients_past_32_bits():
    E, N, K = 1024, 2048, 2056
    counts = [3] + [0] * 500 + [2] + [0] * 521 + [7]
    R = sum(counts)
    assert len(counts) == E and E * N * K > 2 ** 32
    x, dC = _rand((R, K), BF16, 1), _rand((R, N), BF16, 2)
    dW = moe.moe_grouped_gemm_w16_dw(dC, x, None, 1, ru.offsets_of(counts))
    for e, a, b in ((0, 0, 3), (501, 3, 5), (1023, 5, 12)):
        ref, mass = ru.grouped_dw(dC[a:b], x[a:b], [b - a])
        ru.assert_close(dW[e], ref[0], ru.sum_bound(b - a, mass[0]))
    assert sum(int(dW[e].count_nonzero()) for e in range(E) if counts[e] == 0) == 0


# ---- streams, graphs, repeated calls -------------------------------------------------------------------

def _all_ops(x, row_of, W, wq, ws, dC, off, R):
    q, s = moe.moe_i8_quantize(x)
    G = moe.moe_grouped_gemm_w16(x, row_of, 3, W, off, R)
    return [q, s, moe.moe_grouped_gemm_i8(q, s, row_of, 3, wq, ws, off, R), moe.moe_linear_i8(x, wq[0], ws[0]), G,
            moe.moe_grouped_gemm_w16_dx(dC, W, off), moe.moe_grouped_gemm_w16_dw(dC, x, row_of, 3, off), moe.moe_silu_mul(G),
            moe.moe_silu_mul_grad(G, moe.moe_silu_mul(G))]


def _op_inputs(counts, seed):
    N, K, E, R = 144, 208, len(counts), sum(counts)
    x, row_of, _ = _case(counts, 37, K, BF16, seed=seed)
    W, dC = _rand((E, N, K), BF16, seed + 3, K ** -0.5), _rand((R, N), BF16, seed + 4)
    wq, ws = moe.moe_i8_quantize(W.view(-1, K))
    return [x, row_of, W, wq.view(E, N, K), ws.view(E, N), dC, ru.offsets_of(counts), R]


def test_same_inputs_same_bits():
    a = _op_inputs([5, 0, 70, 200], 1)
    first = _all_ops(*a)
    for _ in range(3):
        assert all(torch.equal(p, r) for p, r in zip(first, _all_ops(*a)))


def test_graph_replays_match_eager():
    """Captured once, replayed with other inputs and group sizes in the same buffers, with eager calls between."""
    sets = [_op_inputs(c, s) for c, s in (([5, 0, 70, 200], 1), ([200, 70, 5, 0], 2), ([0, 275, 0, 0], 3))]
    live = [t.clone() if torch.is_tensor(t) else t for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all_ops(*live)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all_ops(*live)
    for n in (0, 1, 2, 1, 0):
        for dst, src in zip(live, sets[n]):
            if torch.is_tensor(dst):
                dst.copy_(src)
        graph.replay()
        want = _all_ops(*sets[n])
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(out, want)), n


def test_two_streams_at_once():
    sets = [_op_inputs([5, 0, 70, 200], 1), _op_inputs([100, 100, 75, 0], 2)]
    want = [_all_ops(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(_all_ops(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(p, r) for p, r in zip(run, want[i]))


def test_given_stream():
    """stream= runs the call there: the outputs made by the wrapper are good once that stream is done."""
    x, row_of, W, wq, ws, dC, off, R = _op_inputs([5, 0, 70, 200], 1)
    want = moe.moe_grouped_gemm_w16(x, row_of, 3, W, off, R), moe.moe_linear_i8(x, wq[0], ws[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = moe.moe_grouped_gemm_w16(x, row_of, 3, W, off, R, stream=st), moe.moe_linear_i8(x, wq[0], ws[0], stream=st)
    st.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(got, want))


def test_binding_refusals():
    """Tensors that would be read wrongly are refused by name."""
    x, logits = _rand((6, 64), BF16, 1), _rand((6, 2), F32, 2)
    W, off = _rand((2, 32, 64), BF16, 3), ru.offsets_of([4, 2])
    q, s = moe.moe_i8_quantize(x)
    wq, ws = moe.moe_i8_quantize(W.view(-1, 64))
    wq, ws = wq.view(2, 32, 64), ws.view(2, 32)
    odd, down = _rand((2, 33, 64), BF16, 4), _rand((2, 64, 16), BF16, 5)
    calls = {
        "w13 must": lambda: moe.moe_ffn_forward_w16(x, logits, odd, down, 1),
        "w13_q must": lambda: moe.moe_ffn_forward_i8(x, logits, torch.zeros((2, 33, 64), dtype=torch.int8, device="cuda"),
                                                     torch.zeros((2, 32), device="cuda"), wq, ws, 1),
        "A must": lambda: moe.moe_grouped_gemm_w16(x.t().contiguous().t(), None, 1, W, off, 6),
        "W must": lambda: moe.moe_grouped_gemm_w16(x, None, 1, W.half(), off, 6),
        "expert_offsets must": lambda: moe.moe_grouped_gemm_w16(x, None, 1, W, off.long(), 6),
        "A has 6 rows": lambda: moe.moe_grouped_gemm_w16(x, None, 1, W, off, 7),
        "a_row_of must hold": lambda: moe.moe_grouped_gemm_w16(x, off, 1, W, off, 7),
        "even N": lambda: moe.moe_grouped_gemm_w16(x, None, 1, W[:, :31].contiguous(), off, 6, epilogue=SILU),
        "As must": lambda: moe.moe_gemm_i8(q, s[:5], wq[0], ws[0]),
        "Ws must": lambda: moe.moe_grouped_gemm_i8(q, s, None, 1, wq, ws[:1], off, 6),
        "C must": lambda: moe.moe_gemm_i8(q, s, wq[0], ws[0], C=torch.empty((6, 32), device="cuda")),
        "dh must": lambda: moe.moe_silu_mul_grad(x, x),
        "G must": lambda: moe.moe_silu_mul(x[:, :63].contiguous()),
        "unknown out_dtype": lambda: moe.moe_gemm_i8(q, s, wq[0], ws[0], out_dtype=9),
        "workspace must": lambda: moe.moe_linear_i8(x, wq[0], ws[0], workspace=torch.empty(4096, device="cuda")),
    }
    for text, call in calls.items():
        with pytest.raises(ValueError, match=text):
            call()


def test_graphs_of_parts_and_layers():
    """Weight gradients in parts, the one-launch linear and the layers, captured together and replayed with other
    inputs."""
    N, K, E, R, T = 136, 144, 2, 2400, 90
    live = {"A": (R, K), "dC": (R, N), "x": (T, 144), "few": (3, K)}
    W, w13, w2 = _rand((E, N, K), BF16, 1, K ** -0.5), _rand((E, 96, 144), BF16, 2, 0.1), _rand((E, 144, 48), BF16, 3, 0.1)
    wq, ws = moe.moe_i8_quantize(W.view(-1, K))
    wq, ws = wq.view(E, N, K), ws.view(E, N)
    w13q, w13s = moe.moe_i8_quantize(w13.view(-1, 144))
    w2q, w2s = moe.moe_i8_quantize(w2.view(-1, 48))
    w13q, w13s, w2q, w2s = w13q.view(E, 96, 144), w13s.view(E, 96), w2q.view(E, 144, 48), w2s.view(E, 144)

    def inputs(seed):
        t = {n: _rand(s, BF16, seed + i) for i, (n, s) in enumerate(live.items())}
        t["logits"] = _rand((T, E), F32, seed + 9)
        t["off"] = ru.offsets_of([1000 + seed, R - 1000 - seed])
        return t

    def calls(t):
        q, s = moe.moe_i8_quantize(t["A"])
        return [moe.moe_grouped_gemm_w16(t["A"], None, 1, W, t["off"], R), moe.moe_grouped_gemm_i8(q, s, None, 1, wq, ws, t["off"], R),
                moe.moe_grouped_gemm_w16_dx(t["dC"], W, t["off"]), moe.moe_grouped_gemm_w16_dw(t["dC"], t["A"], None, 1, t["off"]),
                moe.moe_linear_i8(t["few"], wq[0], ws[0]), moe.moe_linear_i8(t["A"], wq[0], ws[0]),
                moe.moe_ffn_forward_w16(t["x"], t["logits"], w13, w2, 1),
                moe.moe_ffn_forward_i8(t["x"], t["logits"], w13q, w13s, w2q, w2s, 1)]

    assert moe.moe_grouped_gemm_w16_dw_workspace_bytes(R, E, N, K) > 0
    sets = [inputs(s) for s in (1, 200, 777)]
    buf = {n: t.clone() for n, t in sets[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(buf)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:  # each its own outputs and workspaces
        with torch.cuda.graph(g):
            outs.append(calls(buf))
    for n in (0, 1, 2, 1, 0):
        for name, src in sets[n].items():
            buf[name].copy_(src)
        graphs[n % 2].replay()
        want = calls(sets[n])
        graphs[1 - n % 2].replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(p, r) for p, r in zip(out, want)), n
