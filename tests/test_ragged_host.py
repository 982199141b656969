"""Refusals of the ragged products, their layers and SiLU*mul: each call fails before anything is launched, so
these run without a GPU (pointers are never read)."""
import ctypes

import pytest
import torch

import moe_w4a16_grouped_amd as moe

FAKE = 1 << 20
BF16, F16, F32 = 0, 2, 1  # MOE_IN_*
OK, ARG, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4
REFUSALS = [
    # entry, arguments that differ from a call that would be valid, status
    ("moe_i8_quantize", dict(rows=-1), ARG), ("moe_i8_quantize", dict(K=8), ARG), ("moe_i8_quantize", dict(K=72), ARG),
    ("moe_i8_quantize", dict(in_dtype=7), ARG), ("moe_i8_quantize", dict(rows=1 << 26), SHAPE),
    ("moe_i8_quantize", dict(K=1 << 21), SHAPE), ("moe_i8_quantize", dict(x=None), ARG),
    ("moe_i8_quantize", dict(q=FAKE + 8), ALIGN), ("moe_i8_quantize", dict(s=FAKE + 2), ALIGN),
    ("moe_gemm_i8", dict(M=-1), ARG), ("moe_gemm_i8", dict(N=0), ARG), ("moe_gemm_i8", dict(K=72), SHAPE),
    ("moe_gemm_i8", dict(K=(1 << 17) + 16), SHAPE), ("moe_gemm_i8", dict(N=(1 << 20) + 1), SHAPE),
    ("moe_gemm_i8", dict(epilogue=2), ARG), ("moe_gemm_i8", dict(out_dtype=2), ARG),
    ("moe_gemm_i8", dict(epilogue=1, N=63), ARG), ("moe_gemm_i8", dict(epilogue=1, out_dtype=1), ARG),
    ("moe_gemm_i8", dict(Ws=None), ARG), ("moe_gemm_i8", dict(Aq=FAKE + 4), ALIGN), ("moe_gemm_i8", dict(C=FAKE + 4), ALIGN),
    ("moe_linear_i8", dict(in_dtype=3), ARG), ("moe_linear_i8", dict(x=None), ARG), ("moe_linear_i8", dict(workspace=None), ARG),
    ("moe_linear_i8", dict(workspace_bytes=16), WS), ("moe_linear_i8", dict(workspace=FAKE + 8), ALIGN),
    ("moe_linear_i8", dict(x=FAKE + 8), ALIGN), ("moe_linear_i8", dict(T=4, x=FAKE + 8), ALIGN),
    ("moe_linear_i8", dict(T=4, y=None), ARG), ("moe_linear_i8", dict(T=4, Ws=None), ARG), ("moe_linear_i8", dict(T=4, N=0), ARG), ("moe_linear_i8", dict(T=-1), ARG), ("moe_linear_i8", dict(K=24), SHAPE),
    ("moe_grouped_gemm_i8", dict(E=0), ARG), ("moe_grouped_gemm_i8", dict(E=1025), SHAPE),
    ("moe_grouped_gemm_i8", dict(expert_offsets=None), ARG), ("moe_grouped_gemm_i8", dict(a_row_div=0), ARG),
    ("moe_grouped_gemm_i8", dict(R=1 << 26), SHAPE), ("moe_grouped_gemm_i8", dict(a_row_of=FAKE + 2), ALIGN),
    ("moe_grouped_gemm_w16", dict(dtype=1), ARG), ("moe_grouped_gemm_w16", dict(K=12), SHAPE),
    ("moe_grouped_gemm_w16", dict(A=None), ARG), ("moe_grouped_gemm_w16", dict(W=FAKE + 8), ALIGN),
    ("moe_grouped_gemm_w16", dict(epilogue=1, N=65), ARG), ("moe_grouped_gemm_w16", dict(expert_offsets=FAKE + 1), ALIGN),
    ("moe_grouped_gemm_w16_dx", dict(N=12), SHAPE), ("moe_grouped_gemm_w16_dx", dict(out_dtype=3), ARG),
    ("moe_grouped_gemm_w16_dx", dict(dC=None), ARG), ("moe_grouped_gemm_w16_dx", dict(expert_offsets=None), ARG),
    ("moe_grouped_gemm_w16_dw", dict(N=12), SHAPE), ("moe_grouped_gemm_w16_dw", dict(K=12), SHAPE),
    ("moe_grouped_gemm_w16_dw", dict(dW=None, R=0), ARG), ("moe_grouped_gemm_w16_dw", dict(expert_offsets=None, R=0), ARG),
    ("moe_grouped_gemm_w16_dw", dict(dW=FAKE + 4), ALIGN), ("moe_grouped_gemm_w16_dw", dict(dtype=3), ARG),
    ("moe_grouped_gemm_w16_dw", dict(R=8192), WS), ("moe_grouped_gemm_w16_dw", dict(R=8192, workspace=FAKE, workspace_bytes=4096), WS),
    ("moe_grouped_gemm_w16_dw", dict(R=8192, workspace=FAKE + 8, workspace_bytes=1 << 20), ALIGN),
    ("moe_silu_mul", dict(I=12), ARG), ("moe_silu_mul", dict(dtype=1), ARG), ("moe_silu_mul", dict(R=-1), ARG),
    ("moe_silu_mul", dict(h=FAKE + 2), ALIGN), ("moe_silu_mul_grad", dict(dh=None), ARG), ("moe_silu_mul_grad", dict(I=1 << 21), SHAPE),
    ("moe_ffn_forward_i8", dict(H=72), SHAPE), ("moe_ffn_forward_i8", dict(k=9), ARG), ("moe_ffn_forward_i8", dict(w2_s=None), ARG),
    ("moe_ffn_forward_i8", dict(workspace_bytes=16), WS), ("moe_ffn_forward_i8", dict(y=FAKE + 8), ALIGN),
    ("moe_ffn_forward_w16", dict(I=24), SHAPE), ("moe_ffn_forward_w16", dict(w13=None), ARG),
    ("moe_ffn_forward_w16", dict(workspace_bytes=16), WS),
    # no rows: nothing to do (the weight gradients are zeros and need their output)
    ("moe_i8_quantize", dict(rows=0, x=None, q=None, s=None), OK), ("moe_gemm_i8", dict(M=0, Aq=None, C=None), OK),
    ("moe_linear_i8", dict(T=0, x=None, y=None, workspace=None, workspace_bytes=0), OK),
    ("moe_grouped_gemm_i8", dict(R=0, Aq=None, C=None), OK), ("moe_grouped_gemm_w16", dict(R=0, A=None, C=None), OK),
    ("moe_grouped_gemm_w16_dx", dict(R=0, dC=None, dA=None), OK), ("moe_silu_mul", dict(R=0, G=None, h=None), OK),
    ("moe_ffn_forward_i8", dict(T=0), OK), ("moe_ffn_forward_w16", dict(T=0), OK),
]
VALID = {
    "moe_i8_quantize": dict(x=FAKE, in_dtype=BF16, rows=4, K=64, q=FAKE, s=FAKE),
    "moe_gemm_i8": dict(Aq=FAKE, As=FAKE, Wq=FAKE, Ws=FAKE, M=4, N=64, K=64, epilogue=0, C=FAKE, out_dtype=0),
    "moe_linear_i8": dict(x=FAKE, in_dtype=BF16, Wq=FAKE, Ws=FAKE, T=400, N=64, K=64, epilogue=0, y=FAKE, out_dtype=0,
                          workspace=FAKE, workspace_bytes=1 << 20),
    "moe_grouped_gemm_i8": dict(Aq=FAKE, As=FAKE, a_row_of=FAKE, a_row_div=2, Wq=FAKE, Ws=FAKE, expert_offsets=FAKE, R=4, E=8,
                                N=64, K=64, epilogue=0, C=FAKE, out_dtype=0),
    "moe_grouped_gemm_w16": dict(A=FAKE, a_row_of=FAKE, a_row_div=2, W=FAKE, dtype=BF16, expert_offsets=FAKE, R=4, E=8, N=64, K=64,
                                 epilogue=0, C=FAKE, out_dtype=0),
    "moe_grouped_gemm_w16_dx": dict(dC=FAKE, W=FAKE, dtype=F16, expert_offsets=FAKE, R=4, E=8, N=64, K=64, dA=FAKE, out_dtype=1),
    "moe_grouped_gemm_w16_dw": dict(dC=FAKE, A=FAKE, a_row_of=None, a_row_div=1, dtype=F16, expert_offsets=FAKE, R=4, E=8, N=64,
                                    K=64, dW=FAKE, out_dtype=1, workspace=None, workspace_bytes=0),
    "moe_silu_mul": dict(G=FAKE, dtype=BF16, R=4, I=64, h=FAKE),
    "moe_silu_mul_grad": dict(G=FAKE, dh=FAKE, dtype=BF16, R=4, I=64, dG=FAKE),
    "moe_ffn_forward_i8": dict(x=FAKE, logits=FAKE, T=4, H=64, I=64, E=8, k=2, w13_q=FAKE, w13_s=FAKE, w2_q=FAKE, w2_s=FAKE, y=FAKE,
                               ids=None, w=None, workspace=FAKE, workspace_bytes=1 << 30),
    "moe_ffn_forward_w16": dict(x=FAKE, logits=FAKE, T=4, H=64, I=64, E=8, k=2, w13=FAKE, w2=FAKE, y=FAKE, ids=None, w=None,
                                workspace=FAKE, workspace_bytes=1 << 30),
}


@pytest.mark.parametrize("entry,change,status", REFUSALS, ids=lambda v: str(v))
def test_refusals(entry, change, status):
    lib = moe.load()
    args = {**VALID[entry], **change}
    assert set(args) == set(VALID[entry])
    fn = getattr(lib, entry)
    assert fn(*args.values(), None) == status
    assert bool(lib.moe_last_error()) == (status != OK)


def test_workspace_sizes():
    lib = moe.load()
    assert moe.moe_linear_i8_workspace_bytes(77, 2048) >= 77 * 2048 + 77 * 4
    assert moe.moe_linear_i8_workspace_bytes(0, 2048) == moe.moe_linear_i8_workspace_bytes(4, 2048) == 0
    assert moe.moe_linear_i8_workspace_bytes(5, 2048) > 0 and moe.moe_linear_i8_workspace_bytes(17, 16) > 0
    assert moe.moe_linear_i8_workspace_bytes(-1, 2048) == moe.moe_linear_i8_workspace_bytes(5, 24) == 0
    assert moe.moe_grouped_gemm_w16_dw_workspace_bytes(8192, 8, 64, 64) >= 2 * 8 * 64 * 64 * 4
    assert moe.moe_grouped_gemm_w16_dw_workspace_bytes(6400, 256, 1024, 2048) == 0  # enough tiles
    assert moe.moe_grouped_gemm_w16_dw_workspace_bytes(300, 8, 64, 64) == 0         # few rows
    assert moe.moe_grouped_gemm_w16_dw_workspace_bytes(8192, 0, 64, 64) == 0
    T, H, I, E, k = 800, 2048, 512, 256, 8
    R = T * k
    assert moe.moe_ffn_i8_workspace_bytes(T, H, I, E, k) >= T * H + T * 4 + R * I * 3 + R * 4 + R * H * 4
    assert moe.moe_ffn_w16_workspace_bytes(T, H, I, E, k) >= R * I * 2 + R * H * 4
    for f in (moe.moe_ffn_i8_workspace_bytes, moe.moe_ffn_w16_workspace_bytes):
        assert f(4, 2048, 512, 8, 9) == f(4, 2040, 512, 8, 2) == f(-1, 2048, 512, 8, 2) == 0


def test_python_refuses_before_the_library():
    """The binding refuses tensors of other types, shapes or devices (here: of the CPU)."""
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((2, 32, 64), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: moe.moe_i8_quantize(x), lambda: moe.moe_grouped_gemm_w16(x, None, 1, w, off, 4),
                 lambda: moe.moe_grouped_gemm_w16_dx(x, w, off), lambda: moe.moe_grouped_gemm_w16_dw(x, x, None, 1, off),
                 lambda: moe.moe_silu_mul(x), lambda: moe.moe_ffn_forward_w16(x, x, w, w, 1)):
        with pytest.raises(ValueError):
            call()


def test_no_weight_gradient_workspace_for_refused_sizes():
    """0 for every size that the call itself refuses."""
    size = moe.moe_grouped_gemm_w16_dw_workspace_bytes
    assert size(8192, 8, 64, 64) > 0
    assert size(8192, 8, 60, 64) == size(8192, 8, 64, 60) == size(1 << 26, 8, 64, 64) == size(8192, 1025, 64, 64) == 0
    assert size((1 << 26) - 1, 1, 1 << 20, 4096) == 0


def test_no_layer_workspace_for_refused_sizes():
    """0 where one expert's gate_up weights pass 4 GiB, which the layers refuse (int8 and 16-bit elements)."""
    for size, I in ((moe.moe_ffn_i8_workspace_bytes, 1 << 15), (moe.moe_ffn_w16_workspace_bytes, 1 << 14)):
        assert size(4, 1 << 16, I, 8, 2) == 0 and size(4, 1 << 16, I - 16, 8, 2) > 0
