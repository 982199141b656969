"""The norm's codes through the products by expert, as a layer in pieces runs them: norm with the residual -> router on y -> top-k ->
permutation -> the first product on the codes, FP8 and int8, against the products of the same codes in 64 bits."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import moe_w4a16_grouped_amd as moe  # noqa: E402
from tests import ragged_util as ru  # noqa: E402
from tests import test_gpu_f8 as f8  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _pieces(T, E, k, H, quant, block_m):
    x, res = _rand((T, H), BF16, 1), _rand((T, H), BF16, 2, 3.0)
    weight = (torch.rand(H, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") + 0.5).to(BF16)
    s, y, q, scale = moe.moe_rmsnorm_add(x, weight, 1e-6, residual=res, quant=quant)
    assert torch.equal(s, (x.float() + res.float()).to(BF16))
    ids, _ = moe.moe_route_topk(moe.moe_router_logits(y, _rand((E, H), BF16, 4, H ** -0.5)), k)
    al = moe.moe_align(ids, E, block_m)
    order = np.argsort(ids.cpu().numpy().reshape(-1), kind="stable")
    assert np.array_equal(al["sorted_ids"].cpu().numpy()[:T * k], order)
    # codes times scales are y before its rounding, to half a step of the code: int8 1/2 of the scale; E4M3 2^-4 of the value, and
    # 2^-10 of the scale below the normal range.  y itself is off by half a step of bf16, 2^-8, more
    v = q.double() * scale.double()[:, None] if quant == moe.MOE_QUANT_I8 else (
        q.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(128, dim=1))
    step = 0.5 * scale.double()[:, None] if quant == moe.MOE_QUANT_I8 else (
        2.0 ** -4 * y.double().abs() * 1.01 + 2.0 ** -10 * scale.double().repeat_interleave(128, dim=1))
    assert bool(((v - y.double()).abs() <= step * 1.001 + 2.0 ** -8 * 1.001 * y.double().abs()).all())
    return q, scale, al


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T,E,k,H,N,block_m", [(1, 8, 2, 512, 256, 16), (37, 6, 2, 1024, 192, 16), (301, 3, 2, 512, 256, 64), (500, 4, 2, 384, 512, 128)])
def test_fp8(T, E, k, H, N, block_m, silu):
    Aq, As, al = _pieces(T, E, k, H, moe.MOE_QUANT_F8, block_m)
    Wq, Ws = (t.view(E, N, -1) for t in moe.moe_f8_quantize(_rand((E * N, H), F32, 5, H ** -0.5)))
    C = moe.moe_grouped_gemm_f8(Aq, As, al["sorted_ids"], k, Wq, Ws, al["tiles"], al["max_tiles"], al["num_tiles"], block_m,
                                moe.MOE_EPI_SILU_MUL if silu else moe.MOE_EPI_NONE, T * k)
    host = lambda t: np.ascontiguousarray(t.cpu().numpy())
    Aq, As, Wq, Ws, order, offsets = map(host, (Aq, As, Wq, Ws, al["sorted_ids"][:T * k], al["offsets"]))
    G = oracle.grouped_proj_f8(Aq, As, order, k, Wq, Ws, offsets)
    mass = oracle.grouped_proj_f8(Aq & 0x7F, As, order, k, Wq & 0x7F, Ws, offsets)
    err = f8._truncation_bound(Aq, As, order // k, Wq, Ws, offsets) + f8._f8_bound_terms(H) * mass
    got, G, err = C.double().cpu(), torch.from_numpy(G), torch.from_numpy(err)
    if silu:
        assert bool(((got - ru.silu_mul(G)).abs() <= ru.silu_bound(G, err) + U * ru.silu_mul(G).abs() + 1e-30).all())
    else:
        assert bool(((got - G).abs() <= err + 1e-30).all())


@pytest.mark.parametrize("T,E,k,H,N", [(1, 8, 2, 512, 256), (37, 6, 2, 1056, 192), (301, 3, 2, 2048, 528)])
def test_int8(T, E, k, H, N):
    Aq, As, al = _pieces(T, E, k, H, moe.MOE_QUANT_I8, 16)
    Wq, Ws = (t.view(E, N, -1).squeeze(-1) for t in moe.moe_i8_quantize(_rand((E * N, H), F32, 5, H ** -0.5)))
    C = moe.moe_grouped_gemm_i8(Aq, As, al["sorted_ids"], k, Wq, Ws, al["offsets"], T * k, out_dtype=moe.MOE_OUT_F32)
    rows = al["sorted_ids"][:T * k].long() // k
    offsets = al["offsets"].tolist()
    for e in range(E):
        of = rows[offsets[e]:offsets[e + 1]]
        ref = (Aq[of].double() @ Wq[e].double().t()) * As[of].double()[:, None] * Ws[e].double()
        ru.assert_close(C[offsets[e]:offsets[e + 1]], ref, 4 * U * ref.abs())  # exact sums; the scales' product and its product with the sum
