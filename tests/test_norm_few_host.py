"""Refusals of the norm, its gradient and the layer for a few tokens: each call fails before anything is launched, so these
run without a GPU (pointers are never read)."""
import pytest
import torch

import moe_w4a16_grouped_amd as moe

FAKE = 1 << 20
BF16, F16, F32 = 0, 2, 1  # MOE_IN_*
OK, ARG, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4
VALID = {
    "moe_rmsnorm_add": dict(x=FAKE, residual=FAKE, dtype=BF16, weight=FAKE, weight_dtype=F32, eps=1e-6, T=4, H=128, s=FAKE, y=FAKE,
                            quant=2, q=FAKE, q_scale=FAKE),
    "moe_rmsnorm_add_grad": dict(dy=FAKE, s=FAKE, dtype=F16, weight=FAKE, weight_dtype=F16, eps=1e-6, ds=FAKE, T=4, H=64, dx=FAKE,
                                 dweight=FAKE, dweight_dtype=1, workspace=FAKE, workspace_bytes=1 << 20),
    "moe_ffn_few_w16": dict(x=FAKE, logits=FAKE, T=4, H=64, I=64, E=8, k=2, w13=FAKE, w2=FAKE, y=FAKE, ids=None, w=None,
                            workspace=FAKE, workspace_bytes=1 << 20),
    "moe_ffn_few_w8a16": dict(x=FAKE, logits=FAKE, T=4, H=64, I=64, E=8, k=2, w13_q=FAKE, w13_s=FAKE, w2_q=FAKE, w2_s=FAKE, y=FAKE,
                              ids=None, w=None, workspace=FAKE, workspace_bytes=1 << 20),
}
NORM = [
    (dict(dtype=1), ARG), (dict(weight_dtype=2), ARG), (dict(weight_dtype=7), ARG), (dict(eps=0.0), ARG), (dict(eps=-1e-6), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(T=-1), ARG), (dict(H=0), ARG), (dict(T=1 << 26), SHAPE),
    (dict(H=1 << 15), SHAPE),
]
FEW = [
    (dict(T=17), SHAPE), (dict(T=-1), ARG), (dict(k=0), ARG), (dict(k=9), ARG), (dict(k=17, E=64), SHAPE), (dict(E=1025), SHAPE),
    (dict(H=72), SHAPE), (dict(H=0), SHAPE), (dict(H=65552), SHAPE), (dict(I=24), SHAPE), (dict(I=0), SHAPE), (dict(I=(1 << 17) + 16), SHAPE),
    (dict(x=None), ARG), (dict(logits=None), ARG), (dict(y=None), ARG), (dict(workspace=None), ARG), (dict(workspace_bytes=1024), WS),
    (dict(x=FAKE + 8), ALIGN), (dict(y=FAKE + 2), ALIGN), (dict(logits=FAKE + 2), ALIGN), (dict(ids=FAKE + 2), ALIGN), (dict(w=FAKE + 1), ALIGN),
    (dict(workspace=FAKE + 4), ALIGN), (dict(T=0, x=None, y=None, workspace=None), OK),
]
REFUSALS = (
    [("moe_rmsnorm_add", c, st) for c, st in NORM] + [("moe_rmsnorm_add_grad", c, st) for c, st in NORM if c != dict(weight_dtype=2)] + [
        ("moe_rmsnorm_add", dict(quant=3), ARG), ("moe_rmsnorm_add", dict(quant=-1), ARG), ("moe_rmsnorm_add", dict(H=136), SHAPE),
        ("moe_rmsnorm_add", dict(quant=1, H=136), SHAPE), ("moe_rmsnorm_add", dict(quant=0, H=132), SHAPE),
        ("moe_rmsnorm_add", dict(x=None), ARG), ("moe_rmsnorm_add", dict(weight=None), ARG), ("moe_rmsnorm_add", dict(s=None), ARG),
        ("moe_rmsnorm_add", dict(quant=0, y=None), ARG), ("moe_rmsnorm_add", dict(q=None), ARG), ("moe_rmsnorm_add", dict(q_scale=None), ARG),
        ("moe_rmsnorm_add", dict(x=FAKE + 8), ALIGN), ("moe_rmsnorm_add", dict(residual=FAKE + 2), ALIGN),
        ("moe_rmsnorm_add", dict(weight=FAKE + 4), ALIGN), ("moe_rmsnorm_add", dict(s=FAKE + 8), ALIGN), ("moe_rmsnorm_add", dict(y=FAKE + 8), ALIGN),
        ("moe_rmsnorm_add", dict(q=FAKE + 8), ALIGN), ("moe_rmsnorm_add", dict(q_scale=FAKE + 2), ALIGN),
        ("moe_rmsnorm_add", dict(T=0, x=None, s=None, y=None, q=None, q_scale=None), OK),
        ("moe_rmsnorm_add_grad", dict(weight_dtype=0), ARG), ("moe_rmsnorm_add_grad", dict(dweight_dtype=2), ARG),
        ("moe_rmsnorm_add_grad", dict(H=68), SHAPE), ("moe_rmsnorm_add_grad", dict(dy=None), ARG), ("moe_rmsnorm_add_grad", dict(s=None), ARG),
        ("moe_rmsnorm_add_grad", dict(dx=None), ARG), ("moe_rmsnorm_add_grad", dict(dweight=None), ARG),
        ("moe_rmsnorm_add_grad", dict(T=0, dweight=None), ARG), ("moe_rmsnorm_add_grad", dict(workspace=None), ARG),
        ("moe_rmsnorm_add_grad", dict(workspace_bytes=64), WS), ("moe_rmsnorm_add_grad", dict(dy=FAKE + 8), ALIGN),
        ("moe_rmsnorm_add_grad", dict(ds=FAKE + 8), ALIGN), ("moe_rmsnorm_add_grad", dict(dweight=FAKE + 4), ALIGN),
        ("moe_rmsnorm_add_grad", dict(workspace=FAKE + 8), ALIGN),
    ] + [(n, c, st) for n in ("moe_ffn_few_w16", "moe_ffn_few_w8a16") for c, st in FEW] + [
        ("moe_ffn_few_w16", dict(w13=None), ARG), ("moe_ffn_few_w16", dict(w2=FAKE + 8), ALIGN),
        ("moe_ffn_few_w8a16", dict(w13_s=None), ARG), ("moe_ffn_few_w8a16", dict(w2_s=None), ARG), ("moe_ffn_few_w8a16", dict(w2_s=FAKE + 2), ALIGN),
    ])


@pytest.mark.parametrize("entry,change,status", REFUSALS, ids=lambda v: str(v))
def test_refusals(entry, change, status):
    lib = moe.load()
    args = {**VALID[entry], **change}
    assert set(args) == set(VALID[entry])
    assert getattr(lib, entry)(*args.values(), None) == status
    assert bool(lib.moe_last_error()) == (status != OK)


def test_workspace_sizes():
    grad, few = moe.moe_rmsnorm_add_grad_workspace_bytes, moe.moe_ffn_few_workspace_bytes
    assert grad(1, 2048) >= 2048 * 4 and grad(100000, 4096) >= 4096 * 4
    assert grad(100000, 4096) == grad(50000, 4096)  # parts of the rows, no more of them with more rows
    assert grad(0, 64) == grad(-1, 64) == grad(4, 60) == grad(4, 1 << 15) == grad(1 << 26, 64) == 0
    assert few(16, 2048, 768, 128, 8) >= 16 * 8 * 768 * 4
    assert few(16, 8192, 768, 128, 8) <= few(16, 2048, 768, 128, 8)  # groups of 8 tokens
    assert few(0, 2048, 768, 128, 8) == few(17, 2048, 768, 128, 8) == few(4, 2040, 768, 128, 8) == few(4, 2048, 768, 8, 9) == 0
    assert few(4, 2048, 768, 64, 17) == few(4, 65552, 768, 8, 2) == few(4, 2048, 768, 1025, 8) == 0


def test_few_workspace_where_one_expert_passes_four_gib():
    few = moe.moe_ffn_few_workspace_bytes
    assert few(1, 65536, 16384, 2, 1) > 0  # 2 GiB of int8 gate_up weights; bf16 ones are refused by the call
    assert few(1, 65536, 32768, 2, 1) == 0  # 4 GiB of int8 ones: refused by both


def test_python_refuses_before_the_library():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_rmsnorm_add(x, w, 1e-6), lambda: moe.moe_rmsnorm_add_grad(x, x, w, 1e-6),
                 lambda: moe.moe_ffn_few_w16(x, x, x, x, 1), lambda: moe.moe_ffn_few_w8a16(x, x, x, x, x, x, 1)):
        with pytest.raises(ValueError):
            call()


class _Sized:
    """What the binding looks at of a GPU tensor: sizes that a C int does not hold need more memory than a test should take."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = shape, dtype

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("the call went on")


def test_sizes_past_a_c_int_are_refused():
    """2^32 + 8 rows would reach the library as 8, whose results would pass for all."""
    n, w = (1 << 32) + 8, _Sized(64)
    tall, wide, half = _Sized(n, 64), _Sized(1, (1 << 32) + 64), _Sized(1 << 31, 64)
    many = _Sized(1, n, 64), _Sized(1, 64, n // 2)
    q, s = _Sized(n, 64, dtype=torch.int8), _Sized(n, dtype=torch.float32)
    logits = _Sized(1, 1, dtype=torch.float32)
    for call in (lambda: moe.moe_rmsnorm_add(tall, w, 1e-6), lambda: moe.moe_rmsnorm_add(wide, _Sized(wide.shape[1]), 1e-6),
                 lambda: moe.moe_rmsnorm_add(half, w, 1e-6), lambda: moe.moe_rmsnorm_add_grad(tall, tall, w, 1e-6),
                 lambda: moe.moe_ffn_few_w16(_Sized(1, 64), logits, *many, 1), lambda: moe.moe_ffn_few_w16(wide, logits, *many, 1),
                 lambda: moe.moe_ffn_few_w8a16(_Sized(1, 64), logits, _Sized(n, 128, 64, dtype=torch.int8), s, q, s, 1),
                 lambda: moe.moe_i8_quantize(tall), lambda: moe.moe_silu_mul(tall), lambda: moe.moe_gemm_i8(q, s, q, s)):
        with pytest.raises(ValueError, match="at most 2147483647"):
            call()
