"""ctypes binding of libmoe_w4a16.so: argument marshalling only.

Each function has the name of the C entry point it calls, takes torch tensors on the GPU, passes
their data pointers and the current HIP stream, and raises ``MoEError`` on a negative status.  With
``stream=`` the call runs on that stream, to which the tensors made for it belong; the caller
sees to it that the tensors given are ready there, and keeps them until it is done.  No call
builds an autograd graph: results of tensors that require grad carry none.  Every step of the
layer runs in the HIP kernels of the library; there is no fallback of any kind: if the library is
not built, loading fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe_w4a16.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED_SHAPE = -2
MOE_ERR_MISALIGNED = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_HIP = -5
MOE_EPI_NONE = 0
MOE_EPI_SILU_MUL = 1
MOE_OUT_BF16 = 0
MOE_OUT_F32 = 1
MOE_LAYOUT_CANONICAL = 0
MOE_LAYOUT_PACKED = 1
MOE_ACT_ROWS = 0
MOE_ACT_TILED = 1
MOE_IN_BF16 = 0
MOE_IN_F32 = 1
MOE_OUT_F8 = 2
MOE_OUT_F16E = 3
MOE_OUT_H16 = 4
MOE_IN_F16 = 2
MOE_OUT_F16 = 5
MOE_QUANT_NONE = 0
MOE_QUANT_I8 = 1
MOE_QUANT_F8 = 2
MOE_FEW_MAX_TOKENS = 16

_lib = None


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m moe_w4a16_grouped_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    sig = {
        "moe_abi_version": ([], I32),
        "moe_status_string": ([I32], ctypes.c_char_p),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_route_topk": ([P, I32, I32, I32, P, P, P], I32),
        "moe_max_tiles": ([I32, I32, I32, I32], I32),
        "moe_align_workspace_bytes": ([I32, I32, I32], SZ),
        "moe_align": ([P, I32, I32, I32, I32, P, P, P, P, P, I32, P, P, SZ, P], I32),
        "moe_w4_prepack": ([P, P, I32, I32, I32, P, P, P], I32),
        "moe_grouped_gemm_w4a16": ([P, P, I32, P, P, I32, I32, I32, I32, P, I32, P, I32, I32, P, I32, P, P], I32),
        "moe_combine": ([P, I32, P, P, P, P, I32, I32, I32, P, P], I32),
        "moe_x_to_f16": ([P, I32, I32, P, P, P], I32),
        "moe_grouped_gemm_w4f16": ([P, P, P, P, P, I32, P, P, I32, I32, I32, I32, P, I32, P, I32, I32, P, I32, P, P, P],
                                   I32),
        "moe_router_logits": ([P, P, I32, I32, I32, P, P], I32),
        "moe_dense_ffn_workspace_bytes": ([I32, I32, I32], SZ),
        "moe_dense_ffn_w4a16": ([P, I32, I32, I32, P, P, P, P, I32, P, P, SZ, P], I32),
        "moe_ffn_block_workspace_bytes": ([I32, I32, I32, I32, I32, I32], SZ),
        "moe_mx_quantize": ([P, I32, I32, P, P, P], I32),
        "moe_mx_prepack": ([P, P, I32, I32, I32, P, P, P], I32),
        "moe_mx_quantize_tiles": ([P, I32, I32, P, I32, P, I32, P, I32, P, P, P], I32),
        "moe_grouped_gemm_mxfp4": ([P, P, P, I32, P, P, I32, I32, I32, I32, I32, P, I32, P, I32, I32, P, P, I32, P],
                                   I32),
        "moe_ffn_mxfp4_block_m": ([I32, I32, I32, I32, I32], I32),
        "moe_ffn_mxfp4_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_forward_mxfp4": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, I32, P, P, P, P, SZ, P], I32),
        "moe_mx8_quantize": ([P, I32, I32, P, P, P], I32),
        "moe_mx8_quantize_tiles": ([P, I32, I32, P, I32, P, I32, P, I32, P, P, P], I32),
        "moe_grouped_gemm_w4a8": ([P, P, P, I32, P, P, I32, I32, I32, I32, I32, P, I32, P, I32, I32, P, P, I32, P],
                                  I32),
        "moe_ffn_w4a8_block_m": ([I32, I32, I32, I32, I32], I32),
        "moe_ffn_w4a8_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_forward_w4a8": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, I32, P, P, P, P, SZ, P], I32),
        "moe_ffn_block_forward": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, I32, P, P, P, P, I32, P, P, P, P, P,
                                   SZ, P], I32),
        "moe_f8_quantize": ([P, I32, I32, I32, P, P, P], I32),
        "moe_grouped_gemm_f8": ([P, P, P, I32, P, P, I32, I32, I32, P, I32, P, I32, I32, P, P, I32, P], I32),
        "moe_ffn_f8_block_m": ([I32, I32, I32], I32),
        "moe_ffn_f8_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_forward_f8": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_ffn_block_m": ([I32, I32, I32, I32], I32),
        "moe_ffn_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_forward": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, I32, P, P, P, P, SZ, P], I32),
        "moe_i8_quantize": ([P, I32, I32, I32, P, P, P], I32),
        "moe_gemm_i8": ([P, P, P, P, I32, I32, I32, I32, P, I32, P], I32),
        "moe_linear_i8_workspace_bytes": ([I32, I32], SZ),
        "moe_linear_i8": ([P, I32, P, P, I32, I32, I32, I32, P, I32, P, SZ, P], I32),
        "moe_grouped_gemm_i8": ([P, P, P, I32, P, P, P, I32, I32, I32, I32, I32, P, I32, P], I32),
        "moe_ffn_i8_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_forward_i8": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_grouped_gemm_w16": ([P, P, I32, P, I32, P, I32, I32, I32, I32, I32, P, I32, P], I32),
        "moe_grouped_gemm_w16_dx": ([P, P, I32, P, I32, I32, I32, I32, P, I32, P], I32),
        "moe_grouped_gemm_w16_dw_workspace_bytes": ([I32, I32, I32, I32], SZ),
        "moe_grouped_gemm_w16_dw": ([P, P, P, I32, I32, P, I32, I32, I32, I32, P, I32, P, SZ, P], I32),
        "moe_silu_mul": ([P, I32, I32, I32, P, P], I32),
        "moe_silu_mul_grad": ([P, P, I32, I32, I32, P, P], I32),
        "moe_ffn_w16_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_forward_w16": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P], I32),
        "moe_rmsnorm_add": ([P, P, I32, P, I32, ctypes.c_float, I32, I32, P, P, I32, P, P, P], I32),
        "moe_rmsnorm_add_grad_workspace_bytes": ([I32, I32], SZ),
        "moe_rmsnorm_add_grad": ([P, P, I32, P, I32, ctypes.c_float, P, I32, I32, P, P, I32, P, SZ, P], I32),
        "moe_ffn_few_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
        "moe_ffn_few_w16": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P], I32),
        "moe_ffn_few_w8a16": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_ffn_noalloc_scratch_bytes": ([], SZ),
        "moe_ffn_forward_noalloc": ([P, P, I32, I32, I32, I32, I32, P, P, P, P, I32, P, P, P, P], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


EXPORTED = ("moe_abi_version", "moe_status_string", "moe_last_error", "moe_route_topk", "moe_max_tiles",
            "moe_align_workspace_bytes", "moe_align", "moe_w4_prepack", "moe_grouped_gemm_w4a16", "moe_combine",
            "moe_router_logits", "moe_dense_ffn_workspace_bytes", "moe_dense_ffn_w4a16",
            "moe_ffn_block_m", "moe_ffn_workspace_bytes", "moe_ffn_forward", "moe_ffn_block_workspace_bytes",
            "moe_ffn_block_forward", "moe_mx_quantize", "moe_mx_quantize_tiles", "moe_mx_prepack", "moe_grouped_gemm_mxfp4", "moe_ffn_mxfp4_block_m",
            "moe_ffn_mxfp4_workspace_bytes", "moe_ffn_forward_mxfp4", "moe_f8_quantize", "moe_grouped_gemm_f8",
            "moe_ffn_f8_block_m", "moe_ffn_f8_workspace_bytes", "moe_ffn_forward_f8", "moe_mx8_quantize",
            "moe_mx8_quantize_tiles", "moe_grouped_gemm_w4a8", "moe_ffn_w4a8_block_m", "moe_ffn_w4a8_workspace_bytes",
            "moe_ffn_forward_w4a8", "moe_ffn_noalloc_scratch_bytes", "moe_ffn_forward_noalloc", "moe_x_to_f16",
            "moe_grouped_gemm_w4f16", "moe_i8_quantize", "moe_gemm_i8", "moe_linear_i8_workspace_bytes", "moe_linear_i8",
            "moe_grouped_gemm_i8", "moe_ffn_i8_workspace_bytes", "moe_ffn_forward_i8", "moe_grouped_gemm_w16",
            "moe_grouped_gemm_w16_dx", "moe_grouped_gemm_w16_dw_workspace_bytes", "moe_grouped_gemm_w16_dw", "moe_silu_mul", "moe_silu_mul_grad",
            "moe_ffn_w16_workspace_bytes", "moe_ffn_forward_w16", "moe_rmsnorm_add", "moe_rmsnorm_add_grad_workspace_bytes",
            "moe_rmsnorm_add_grad", "moe_ffn_few_workspace_bytes", "moe_ffn_few_w16", "moe_ffn_few_w8a16")


def _check(status: int):
    if status != MOE_OK:
        lib = load()
        raise MoEError(status, f"{lib.moe_status_string(status).decode()}: {lib.moe_last_error().decode()}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, dev, stream=None, keep=True, like=None):
    """Memory that a wrapper makes for its call belongs to the stream of the call: a block that the current stream's
    allocator gives may still be in use by work queued there, which another stream does not wait for.  keep: the caller
    gets the tensor, and may use and free it on the current stream too (once that waits for the given one).  like: a
    tensor of the shape and device, from which torch makes another faster."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else torch.empty_like(like, dtype=dtype)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if keep:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _req(t, dtype, name):
    ok = t.element_size() == 2 if dtype == "16bit" else t.dtype == dtype
    if not ok or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor (got {t.dtype}, {t.device})")
    return t


# ---- entry points ----------------------------------------------------------------------------------

def moe_max_tiles(T: int, k: int, E: int, block_m: int) -> int:
    return int(load().moe_max_tiles(T, k, E, block_m))


def moe_align_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(load().moe_align_workspace_bytes(T, k, E))


def moe_ffn_block_m(T: int, E: int, k: int, weight_layout: int = 0) -> int:
    return int(load().moe_ffn_block_m(T, E, k, weight_layout))


def moe_ffn_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_workspace_bytes(T, H, I, E, k))


def moe_route_topk(logits: torch.Tensor, k: int, topk_ids=None, topk_w=None, stream=None):
    """logits fp32 [T, E] -> (topk_ids int32 [T, k], topk_w fp32 [T, k])."""
    _req(logits, torch.float32, "logits")
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = _empty((T, k), torch.int32, logits.device, stream)
    if topk_w is None:
        topk_w = _empty((T, k), torch.float32, logits.device, stream)
    _check(load().moe_route_topk(_p(logits), T, E, k, _p(topk_ids), _p(topk_w), _stream(stream)))
    return topk_ids, topk_w


def moe_align(topk_ids: torch.Tensor, E: int, block_m: int, stream=None, max_tiles: int = None) -> dict:
    """topk_ids int32 [T, k] -> dict of device tensors (counts, offsets, sorted_ids, inv_perm, tiles,
    num_tiles) and the tile capacity ``max_tiles`` (default: moe_max_tiles; a larger capacity may be
    given)."""
    _req(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    dev = topk_ids.device
    R = T * k
    if max_tiles is None:
        max_tiles = moe_max_tiles(T, k, E, block_m)
    out = dict(
        counts=_empty(E, torch.int32, dev, stream),
        offsets=_empty(E + 1, torch.int32, dev, stream),
        sorted_ids=_empty(max(R, 1), torch.int32, dev, stream),
        inv_perm=_empty(max(R, 1), torch.int32, dev, stream),
        tiles=_empty((max(max_tiles, 1), 3), torch.int32, dev, stream),
        num_tiles=_empty(1, torch.int32, dev, stream),
    )
    wsb = moe_align_workspace_bytes(T, k, E)
    ws = _empty(max(wsb, 16), torch.uint8, dev, stream, keep=False) if wsb else None
    _check(load().moe_align(_p(topk_ids), T, k, E, block_m, _p(out["counts"]), _p(out["offsets"]),
                            _p(out["sorted_ids"]), _p(out["inv_perm"]), _p(out["tiles"]), max_tiles,
                            _p(out["num_tiles"]), _p(ws), wsb, _stream(stream)))
    out["max_tiles"] = max_tiles
    out["_workspace"] = ws
    return out


def moe_w4_prepack(w_q, w_s, packed_q=None, packed_s=None, stream=None):
    """Canonical [E, N, K/2] codes + [E, N, K/32] scales -> the same tensors in the packed layout
    (returned with the canonical shapes, which describe their sizes, not their element order)."""
    _req(w_q, torch.uint8, "w_q")
    _req(w_s, "16bit", "w_s")
    E, N, K2 = w_q.shape
    if packed_q is None:
        packed_q = _empty(w_q.shape, w_q.dtype, w_q.device, stream)
    if packed_s is None:
        packed_s = _empty(w_s.shape, w_s.dtype, w_s.device, stream)
    _check(load().moe_w4_prepack(_p(w_q), _p(w_s), E, N, 2 * K2, _p(packed_q), _p(packed_s), _stream(stream)))
    return packed_q, packed_s


def moe_grouped_gemm_w4a16(A, a_row_of, a_row_div: int, Wq, Ws, tiles, max_tiles: int, num_tiles,
                           block_m: int, epilogue: int, out_rows: int, out_dtype: int = MOE_OUT_BF16,
                           C=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL, C_side=None):
    """Grouped W4A16 GEMM over the tile list; returns C ([out_rows, N] or [out_rows, N/2]), or
    (C fp16, C_side fp32 [out_rows, ceil(N/8)]) for MOE_OUT_F16E."""
    _req(A, "16bit", "A")
    _req(Wq, torch.uint8, "Wq")
    E, N, K2 = Wq.shape
    K = 2 * K2
    ncols = N // 2 if epilogue == MOE_EPI_SILU_MUL else N
    if C is None:
        dt = {MOE_OUT_F32: torch.float32, MOE_OUT_F16E: torch.float16}.get(out_dtype, torch.bfloat16)
        C = _empty((out_rows, ncols), dt, A.device, stream)
    if out_dtype == MOE_OUT_F16E and C_side is None:
        C_side = _empty((out_rows, (ncols + 7) // 8), torch.float32, A.device, stream)
    _check(load().moe_grouped_gemm_w4a16(_p(A), _p(a_row_of), a_row_div, _p(Wq), _p(Ws), weight_layout, E, N, K,
                                         _p(tiles),
                                         max_tiles, _p(num_tiles), block_m, epilogue, _p(C), out_dtype, _p(C_side),
                                         _stream(stream)))
    return (C, C_side) if out_dtype == MOE_OUT_F16E else C


def moe_x_to_f16(x, x16=None, x_exp=None, stream=None):
    """bf16 x [T, H] -> (fp16 x16 [T, H], int32 row exponents [T]): x16 = fp16(x * 2^-x_exp)."""
    _req(x, "16bit", "x")
    T, H = x.shape
    if x16 is None:
        x16 = _empty((T, H), torch.float16, x.device, stream)
    if x_exp is None:
        x_exp = _empty((T,), torch.int32, x.device, stream)
    _check(load().moe_x_to_f16(_p(x), T, H, _p(x16), _p(x_exp), _stream(stream)))
    return x16, x_exp


def moe_grouped_gemm_w4f16(A, a_row_exp, a_exps, a_row_of, a_row_div: int, Wq, Ws, tiles, max_tiles: int,
                           num_tiles, block_m: int, epilogue: int, out_rows: int, out_dtype: int, C=None, C_aux=None,
                           C_aux2=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL):
    """Grouped GEMM of the exact fp16 path (fp16 activations with exponents).  a_exps: None or the
    (flags, row exponents) pair a SILU_MUL call returned for h.  Returns (h fp16, (flags, row
    exponents)) for SILU_MUL, (C fp16, side fp32) for MOE_OUT_F16E, or C fp32 for MOE_OUT_F32."""
    _req(A, "16bit", "A")
    _req(Wq, torch.uint8, "Wq")
    E, N, K2 = Wq.shape
    K = 2 * K2
    ncols = N // 2 if epilogue == MOE_EPI_SILU_MUL else N
    if C is None:
        C = _empty((out_rows, ncols), torch.float32 if out_dtype == MOE_OUT_F32 else torch.float16, A.device, stream)
    if out_dtype == MOE_OUT_H16:
        if C_aux is None:
            C_aux = _empty((max(max_tiles, 1), (ncols + 31) // 32), torch.uint8, A.device, stream)
        if C_aux2 is None:
            C_aux2 = _empty((out_rows, (ncols + 31) // 32), torch.uint8, A.device, stream)
    elif C_aux is None and out_dtype == MOE_OUT_F16E:
        C_aux = _empty((out_rows, (ncols + 7) // 8), torch.float32, A.device, stream)
    bf, be = (None, None) if a_exps is None else a_exps
    _check(load().moe_grouped_gemm_w4f16(_p(A), _p(a_row_exp), _p(bf), _p(be), _p(a_row_of), a_row_div, _p(Wq), _p(Ws),
                                         weight_layout, E, N, K, _p(tiles), max_tiles, _p(num_tiles), block_m, epilogue,
                                         _p(C), out_dtype, _p(C_aux), _p(C_aux2), _stream(stream)))
    if out_dtype == MOE_OUT_F32:
        return C
    return (C, (C_aux, C_aux2)) if out_dtype == MOE_OUT_H16 else (C, C_aux)


def moe_combine(O, inv_perm, topk_w, y=None, stream=None, shared=None, O_side=None):
    """O fp32 [T*k, H], or fp16 [T*k, H] with side values O_side fp32 [T*k, H/8] (MOE_OUT_F16E),
    inv_perm int32 [T*k], topk_w fp32 [T, k] (+ shared fp32 [T, H]) -> y bf16 [T, H]."""
    if O.dtype == torch.float16:
        if O_side is None:
            raise ValueError("fp16 O needs its side values O_side")
        _req(O_side, torch.float32, "O_side")
        o_dtype = MOE_OUT_F16E
    else:
        _req(O, torch.float32, "O")
        o_dtype = MOE_OUT_F32
    if shared is not None:
        _req(shared, torch.float32, "shared")
    T, k = topk_w.shape
    H = O.shape[1]
    if y is None:
        y = _empty((T, H), torch.bfloat16, O.device, stream)
    _check(load().moe_combine(_p(O), o_dtype, _p(O_side) if o_dtype == MOE_OUT_F16E else None, _p(inv_perm),
                              _p(topk_w), _p(shared), T, k, H, _p(y), _stream(stream)))
    return y


def moe_router_logits(x, w_router, logits=None, stream=None):
    """x bf16 [T, H], w_router bf16 [E, H] -> logits fp32 [T, E]."""
    _req(x, "16bit", "x")
    _req(w_router, "16bit", "w_router")
    T, H = x.shape
    E = w_router.shape[0]
    if logits is None:
        logits = _empty((T, E), torch.float32, x.device, stream)
    _check(load().moe_router_logits(_p(x), _p(w_router), T, H, E, _p(logits), _stream(stream)))
    return logits


def moe_dense_ffn_workspace_bytes(T: int, H: int, I: int) -> int:
    return int(load().moe_dense_ffn_workspace_bytes(T, H, I))


def moe_dense_ffn_w4a16(x, w13_q, w13_s, w2_q, w2_s, out=None, workspace=None, stream=None,
                        weight_layout: int = MOE_LAYOUT_CANONICAL):
    """One dense SwiGLU expert on every token: x bf16 [T, H], w13_q [2I, H/2], w2_q [H, I/2] -> fp32 [T, H]."""
    _req(x, "16bit", "x")
    T, H = x.shape
    I = w13_q.shape[-2] // 2
    if out is None:
        out = _empty((T, H), torch.float32, x.device, stream)
    wsb = moe_dense_ffn_workspace_bytes(T, H, I)
    if workspace is None:
        workspace = _empty(max(wsb, 256), torch.uint8, x.device, stream, keep=False)
    _check(load().moe_dense_ffn_w4a16(_p(x), T, H, I, _p(w13_q), _p(w13_s), _p(w2_q), _p(w2_s), weight_layout,
                                      _p(out), _p(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream)))
    return out


def moe_ffn_block_workspace_bytes(T: int, H: int, I: int, E: int, k: int, Is: int = 0) -> int:
    return int(load().moe_ffn_block_workspace_bytes(T, H, I, E, k, Is))


def moe_ffn_block_forward(x, w_router, w13_q, w13_s, w2_q, w2_s, k: int, shared=None, y=None, logits_out=None,
                          topk_ids_out=None, topk_w_out=None, workspace=None, stream=None,
                          weight_layout: int = MOE_LAYOUT_CANONICAL):
    """Whole MoE block: router gate, optional shared expert ``shared = (w13s_q, w13s_s, w2s_q, w2s_s)``,
    routed experts and combine.  x bf16 [T, H], w_router bf16 [E, H] -> y bf16 [T, H]."""
    _req(x, "16bit", "x")
    T, H = x.shape
    E, N13, _ = w13_q.shape
    I = N13 // 2
    if shared is None:
        Is, sh = 0, (None, None, None, None)
    else:
        Is, sh = shared[0].shape[-2] // 2, shared
    if y is None:
        y = _empty((T, H), torch.bfloat16, x.device, stream)
    wsb = moe_ffn_block_workspace_bytes(T, H, I, E, k, Is)
    if workspace is None:
        workspace = _empty(max(wsb, 256), torch.uint8, x.device, stream, keep=False)
    _check(load().moe_ffn_block_forward(_p(x), _p(w_router), T, H, I, E, k, _p(w13_q), _p(w13_s), _p(w2_q),
                                        _p(w2_s), Is, *(_p(t) for t in sh), weight_layout, _p(y), _p(logits_out),
                                        _p(topk_ids_out), _p(topk_w_out), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


def moe_ffn_forward(x, router_logits, w13_q, w13_s, w2_q, w2_s, k: int, y=None, topk_ids_out=None,
                    topk_w_out=None, workspace=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL):
    """Whole layer: x bf16 [T, H], logits fp32 [T, E], weights in the W4 group-32 format -> y bf16."""
    T, H = x.shape
    E, N13, _ = w13_q.shape
    I = N13 // 2
    if y is None:
        y = _empty((T, H), torch.bfloat16, x.device, stream)
    wsb = moe_ffn_workspace_bytes(T, H, I, E, k)
    if workspace is None:
        workspace = _empty(max(wsb, 256), torch.uint8, x.device, stream, keep=False)
    _check(load().moe_ffn_forward(_p(x), _p(router_logits), T, H, I, E, k, _p(w13_q), _p(w13_s), _p(w2_q),
                                  _p(w2_s), weight_layout, _p(y), _p(topk_ids_out), _p(topk_w_out), _p(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


def moe_ffn_noalloc_scratch_bytes() -> int:
    return int(load().moe_ffn_noalloc_scratch_bytes())


def moe_ffn_forward_noalloc(x, router_logits, w13_q, w13_s, w2_q, w2_s, k: int, y=None, topk_ids_out=None,
                            topk_w_out=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL):
    """moe_ffn_forward working in the library's static device scratch (the C call allocates nothing;
    y is allocated here only when the caller passes none)."""
    T, H = x.shape
    E, N13, _ = w13_q.shape
    I = N13 // 2
    if y is None:
        y = _empty((T, H), torch.bfloat16, x.device, stream)
    _check(load().moe_ffn_forward_noalloc(_p(x), _p(router_logits), T, H, I, E, k, _p(w13_q), _p(w13_s), _p(w2_q),
                                          _p(w2_s), weight_layout, _p(y), _p(topk_ids_out), _p(topk_w_out),
                                          _stream(stream)))
    return y


# ---- MXFP4 (W4A4) ----------------------------------------------------------------------------------

def moe_mx_quantize(x, q=None, s=None, stream=None):
    """x bf16 [rows, K] -> (codes uint8 [rows, K/2], scale bytes uint8 [rows, K/32])."""
    _req(x, "16bit", "x")
    rows, K = x.shape
    if q is None:
        q = _empty((rows, K // 2), torch.uint8, x.device, stream)
    if s is None:
        s = _empty((rows, K // 32), torch.uint8, x.device, stream)
    _check(load().moe_mx_quantize(_p(x), rows, K, _p(q), _p(s), _stream(stream)))
    return q, s


def moe_mx_prepack(w_q, w_e, packed_q=None, packed_e=None, stream=None):
    """Canonical MXFP4 weights (codes [E, N, K/2], scale bytes [E, N, K/32]) -> the packed layout
    (returned with the canonical shapes, which describe sizes, not element order)."""
    _req(w_q, torch.uint8, "w_q")
    _req(w_e, torch.uint8, "w_e")
    E, N, K2 = w_q.shape
    if packed_q is None:
        packed_q = _empty(w_q.shape, w_q.dtype, w_q.device, stream)
    if packed_e is None:
        packed_e = _empty(w_e.shape, w_e.dtype, w_e.device, stream)
    _check(load().moe_mx_prepack(_p(w_q), _p(w_e), E, N, 2 * K2, _p(packed_q), _p(packed_e), _stream(stream)))
    return packed_q, packed_e


def moe_mx_quantize_tiles(x, a_row_of, a_row_div: int, tiles, max_tiles: int, num_tiles, block_m: int, q=None, s=None,
                          stream=None):
    """x bf16 [T, K] -> tile-blocked codes (uint8 [max_tiles * block_m, K/2]) and scale bytes
    (uint8 [max_tiles * block_m, K/32]) of the tile list (shapes give sizes, not element order)."""
    _req(x, "16bit", "x")
    T, K = x.shape
    rows = max(max_tiles, 1) * block_m
    if q is None:
        q = _empty((rows, K // 2), torch.uint8, x.device, stream)
    if s is None:
        s = _empty((rows, K // 32), torch.uint8, x.device, stream)
    if q.numel() < rows * (K // 2) or s.numel() < rows * (K // 32):
        raise ValueError(f"tile-blocked activations need {rows} rows (max_tiles * block_m)")
    _check(load().moe_mx_quantize_tiles(_p(x), T, K, _p(a_row_of), a_row_div, _p(tiles), max_tiles, _p(num_tiles),
                                        block_m, _p(q), _p(s), _stream(stream)))
    return q, s


def moe_grouped_gemm_mxfp4(Aq, As, a_row_of, a_row_div: int, Wq, We, tiles, max_tiles: int, num_tiles,
                           block_m: int, epilogue: int, out_rows: int, out_dtype: int = MOE_OUT_F32, C=None,
                           Cs=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL,
                           act_layout: int = MOE_ACT_ROWS):
    """Grouped MXFP4 GEMM over the tile list.  NONE: returns C [out_rows, N]; SILU_MUL: returns the
    quantized h as (codes [out_rows, N/4], scale bytes [out_rows, N/64]); with act_layout TILED the
    h buffers must hold max_tiles * block_m rows (tile-blocked)."""
    _req(Aq, torch.uint8, "Aq")
    _req(Wq, torch.uint8, "Wq")
    E, N, K2 = Wq.shape
    K = 2 * K2
    dev = Aq.device
    if act_layout == MOE_ACT_TILED and epilogue == MOE_EPI_SILU_MUL:
        out_rows = max(out_rows, max(max_tiles, 1) * block_m)  # h is written tile-blocked
    if epilogue == MOE_EPI_SILU_MUL:
        if C is None:
            C = _empty((out_rows, N // 4), torch.uint8, dev, stream)
        if Cs is None:
            Cs = _empty((out_rows, N // 64), torch.uint8, dev, stream)
    elif C is None:
        C = _empty((out_rows, N), torch.float32 if out_dtype == MOE_OUT_F32 else torch.bfloat16, dev, stream)
    if act_layout == MOE_ACT_TILED and epilogue == MOE_EPI_SILU_MUL:
        need = max(max_tiles, 1) * block_m
        if C.shape[0] < need or Cs.shape[0] < need:
            raise ValueError(f"tile-blocked h needs {need} rows (max_tiles * block_m), got {C.shape[0]}")
    _check(load().moe_grouped_gemm_mxfp4(_p(Aq), _p(As), _p(a_row_of), a_row_div, _p(Wq), _p(We), weight_layout,
                                         act_layout, E, N, K, _p(tiles),
                                         max_tiles, _p(num_tiles), block_m, epilogue, _p(C), _p(Cs), out_dtype,
                                         _stream(stream)))
    return (C, Cs) if epilogue == MOE_EPI_SILU_MUL else C


def moe_ffn_mxfp4_block_m(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_mxfp4_block_m(T, H, I, E, k))


def moe_ffn_mxfp4_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_mxfp4_workspace_bytes(T, H, I, E, k))


def moe_ffn_forward_mxfp4(x, router_logits, w13_q, w13_e, w2_q, w2_e, k: int, y=None, topk_ids_out=None,
                          topk_w_out=None, workspace=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL):
    """Whole MXFP4 (W4A4) layer: x bf16 [T, H], logits fp32 [T, E], MXFP4 weights -> y bf16 [T, H]."""
    _req(x, "16bit", "x")
    T, H = x.shape
    E, N13, _ = w13_q.shape
    I = N13 // 2
    if y is None:
        y = _empty((T, H), torch.bfloat16, x.device, stream)
    wsb = moe_ffn_mxfp4_workspace_bytes(T, H, I, E, k)
    if workspace is None:
        workspace = _empty(max(wsb, 256), torch.uint8, x.device, stream, keep=False)
    _check(load().moe_ffn_forward_mxfp4(_p(x), _p(router_logits), T, H, I, E, k, _p(w13_q), _p(w13_e), _p(w2_q),
                                        _p(w2_e), weight_layout, _p(y), _p(topk_ids_out), _p(topk_w_out), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


# ---- W4A8 (MXFP8 activations on MXFP4 weights) ------------------------------------------------------

def moe_mx8_quantize(x, q=None, s=None, stream=None):
    """x bf16 [rows, K] -> MXFP8 (codes uint8 [rows, K], scale bytes uint8 [rows, K/32])."""
    _req(x, "16bit", "x")
    rows, K = x.shape
    if q is None:
        q = _empty((rows, K), torch.uint8, x.device, stream)
    if s is None:
        s = _empty((rows, K // 32), torch.uint8, x.device, stream)
    _check(load().moe_mx8_quantize(_p(x), rows, K, _p(q), _p(s), _stream(stream)))
    return q, s


def moe_mx8_quantize_tiles(x, a_row_of, a_row_div: int, tiles, max_tiles: int, num_tiles, block_m: int, q=None,
                           s=None, stream=None):
    """x bf16 [T, K] -> tile-blocked MXFP8 codes [max_tiles * block_m, K] and scale bytes [.., K/32]."""
    _req(x, "16bit", "x")
    T, K = x.shape
    rows = max(max_tiles, 1) * block_m
    if q is None:
        q = _empty((rows, K), torch.uint8, x.device, stream)
    if s is None:
        s = _empty((rows, K // 32), torch.uint8, x.device, stream)
    _check(load().moe_mx8_quantize_tiles(_p(x), T, K, _p(a_row_of), a_row_div, _p(tiles), max_tiles, _p(num_tiles),
                                         block_m, _p(q), _p(s), _stream(stream)))
    return q, s


def moe_grouped_gemm_w4a8(Aq, As, a_row_of, a_row_div: int, Wq, We, tiles, max_tiles: int, num_tiles,
                          block_m: int, epilogue: int, out_rows: int, out_dtype: int = MOE_OUT_F32, C=None,
                          Cs=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL,
                          act_layout: int = MOE_ACT_ROWS):
    """Grouped W4A8 GEMM over the tile list (MXFP8 activations).  NONE: returns C [out_rows, N];
    SILU_MUL: returns the MXFP8 h as (codes [out_rows, N/2], scale bytes [out_rows, N/64]); with
    act_layout TILED the h buffers hold max_tiles * block_m rows (tile-blocked)."""
    _req(Aq, torch.uint8, "Aq")
    _req(Wq, torch.uint8, "Wq")
    E, N, K2 = Wq.shape
    K = 2 * K2
    dev = Aq.device
    if act_layout == MOE_ACT_TILED and epilogue == MOE_EPI_SILU_MUL:
        out_rows = max(out_rows, max(max_tiles, 1) * block_m)  # h is written tile-blocked
    if epilogue == MOE_EPI_SILU_MUL:
        if C is None:
            C = _empty((out_rows, N // 2), torch.uint8, dev, stream)
        if Cs is None:
            Cs = _empty((out_rows, N // 64), torch.uint8, dev, stream)
    elif C is None:
        C = _empty((out_rows, N), torch.float32 if out_dtype == MOE_OUT_F32 else torch.bfloat16, dev, stream)
    _check(load().moe_grouped_gemm_w4a8(_p(Aq), _p(As), _p(a_row_of), a_row_div, _p(Wq), _p(We), weight_layout,
                                        act_layout, E, N, K, _p(tiles), max_tiles, _p(num_tiles), block_m, epilogue,
                                        _p(C), _p(Cs), out_dtype, _stream(stream)))
    return (C, Cs) if epilogue == MOE_EPI_SILU_MUL else C


def moe_ffn_w4a8_block_m(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_w4a8_block_m(T, H, I, E, k))


def moe_ffn_w4a8_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_w4a8_workspace_bytes(T, H, I, E, k))


def moe_ffn_forward_w4a8(x, router_logits, w13_q, w13_e, w2_q, w2_e, k: int, y=None, topk_ids_out=None,
                         topk_w_out=None, workspace=None, stream=None, weight_layout: int = MOE_LAYOUT_CANONICAL):
    """Whole W4A8 layer: x bf16 [T, H], logits fp32 [T, E], MXFP4 weights -> y bf16 [T, H]."""
    _req(x, "16bit", "x")
    T, H = x.shape
    E, N13, _ = w13_q.shape
    I = N13 // 2
    if y is None:
        y = _empty((T, H), torch.bfloat16, x.device, stream)
    wsb = moe_ffn_w4a8_workspace_bytes(T, H, I, E, k)
    if workspace is None:
        workspace = _empty(max(wsb, 256), torch.uint8, x.device, stream, keep=False)
    _check(load().moe_ffn_forward_w4a8(_p(x), _p(router_logits), T, H, I, E, k, _p(w13_q), _p(w13_e), _p(w2_q),
                                       _p(w2_e), weight_layout, _p(y), _p(topk_ids_out), _p(topk_w_out), _p(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


# ---- FP8 (W8A8, per-1x128) -------------------------------------------------------------------------

def moe_f8_quantize(x, q=None, s=None, stream=None):
    """x bf16 or fp32 [rows, K] -> (E4M3 codes uint8 [rows, K], fp32 scales [rows, K/128])."""
    if x.dtype == torch.float32:
        in_dtype = MOE_IN_F32
    else:
        _req(x, "16bit", "x")
        in_dtype = MOE_IN_BF16
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")
    rows, K = x.shape
    if q is None:
        q = _empty((rows, K), torch.uint8, x.device, stream)
    if s is None:
        s = _empty((rows, K // 128), torch.float32, x.device, stream)
    _check(load().moe_f8_quantize(_p(x), in_dtype, rows, K, _p(q), _p(s), _stream(stream)))
    return q, s


def moe_grouped_gemm_f8(Aq, As, a_row_of, a_row_div: int, Wq, Ws, tiles, max_tiles: int, num_tiles, block_m: int,
                        epilogue: int, out_rows: int, out_dtype: int = MOE_OUT_F32, C=None, Cs=None, stream=None):
    """Grouped FP8 GEMM over the tile list.  NONE: returns C [out_rows, N] (fp32 or bf16); SILU_MUL:
    returns h fp32 [out_rows, N/2], or with out_dtype MOE_OUT_F8 the quantized h as (codes uint8
    [out_rows, N/2], scales fp32 [out_rows, N/256])."""
    _req(Aq, torch.uint8, "Aq")
    _req(Wq, torch.uint8, "Wq")
    E, N, K = Wq.shape
    if out_dtype == MOE_OUT_F8:
        if C is None:
            C = _empty((out_rows, N // 2), torch.uint8, Aq.device, stream)
        if Cs is None:
            Cs = _empty((out_rows, max(N // 256, 1)), torch.float32, Aq.device, stream)
    elif C is None:
        cols = N // 2 if epilogue == MOE_EPI_SILU_MUL else N
        dt = torch.float32 if out_dtype == MOE_OUT_F32 else torch.bfloat16
        C = _empty((out_rows, cols), dt, Aq.device, stream)
    _check(load().moe_grouped_gemm_f8(_p(Aq), _p(As), _p(a_row_of), a_row_div, _p(Wq), _p(Ws), E, N, K, _p(tiles),
                                      max_tiles, _p(num_tiles), block_m, epilogue, _p(C), _p(Cs), out_dtype,
                                      _stream(stream)))
    return (C, Cs) if out_dtype == MOE_OUT_F8 else C


def moe_ffn_f8_block_m(T: int, E: int, k: int) -> int:
    return int(load().moe_ffn_f8_block_m(T, E, k))


def moe_ffn_f8_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_f8_workspace_bytes(T, H, I, E, k))


def moe_ffn_forward_f8(x, router_logits, w13_q, w13_s, w2_q, w2_s, k: int, y=None, topk_ids_out=None,
                       topk_w_out=None, workspace=None, stream=None):
    """Whole FP8 (W8A8, per-1x128) layer: x bf16 [T, H], logits fp32 [T, E], E4M3 weights with fp32
    scales -> y bf16 [T, H]."""
    _req(x, "16bit", "x")
    T, H = x.shape
    E, N13, _ = w13_q.shape
    I = N13 // 2
    if y is None:
        y = _empty((T, H), torch.bfloat16, x.device, stream)
    wsb = moe_ffn_f8_workspace_bytes(T, H, I, E, k)
    if workspace is None:
        workspace = _empty(max(wsb, 256), torch.uint8, x.device, stream, keep=False)
    _check(load().moe_ffn_forward_f8(_p(x), _p(router_logits), T, H, I, E, k, _p(w13_q), _p(w13_s), _p(w2_q),
                                     _p(w2_s), _p(y), _p(topk_ids_out), _p(topk_w_out), _p(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


# ---- ragged products: INT8 (W8A8, per token and channel) and 16-bit expert weights ---------------------

_IN = {torch.bfloat16: MOE_IN_BF16, torch.float16: MOE_IN_F16, torch.float32: MOE_IN_F32}
_OUT = {torch.bfloat16: MOE_OUT_BF16, torch.float16: MOE_OUT_F16, torch.float32: MOE_OUT_F32}
_OUT_DTYPE = {v: k for k, v in _OUT.items()}
_W16 = (torch.bfloat16, torch.float16)
_I8, _F32, _INT32, _U8, _BF16 = (torch.int8,), (torch.float32,), (torch.int32,), (torch.uint8,), (torch.bfloat16,)
_ACT = tuple(_IN)


_C_INT = 2 ** 31 - 1  # ctypes would pass larger sizes on without their upper bits


def _need(t, dtypes, shape, name, dev=None):
    """A contiguous GPU tensor of one of the dtypes and of this shape (None = any size that a C int holds, ... = any that the
    call is not told or takes in 64 bits), on dev."""
    s = t.shape
    if t.dtype in dtypes and t.is_cuda and t.is_contiguous() and (dev is None or t.device == dev):
        if len(s) == len(shape):
            for got, want in zip(s, shape):
                if want is None:
                    if got > _C_INT:
                        raise ValueError(f"{name} has a dimension of {got} (at most {_C_INT})")
                elif got != want and want is not ...:
                    break
            else:
                return s
        raise ValueError(f"{name} must have the shape {shape} (got {tuple(s)})")
    raise ValueError(f"{name} must be a contiguous {' or '.join(str(x) for x in dtypes)} CUDA tensor"
                     f"{'' if dev is None else f' on {dev}'} (got {t.dtype}, {t.device})")


def _call(fn, dev, stream, made, *args):
    """Calls a C entry point on the tensors' device and stream.  made: the call's outputs and workspaces, whose memory
    is kept until a given stream is done (those that the caller gave may belong to another one)."""
    index = dev.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        if stream.device != dev:
            raise ValueError(f"stream is of {stream.device}, the tensors of {dev}")
        raw = stream.cuda_stream
        for t in made:
            if t is not None:
                t.record_stream(stream)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != MOE_OK:
        _check(status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _out(made, shape, out_dtype, dev, name, stream):
    """The caller's output, checked, or a new one of out_dtype; a call's out_dtype defaults to bf16."""
    dt = _OUT_DTYPE.get(out_dtype)
    if dt is None:
        raise ValueError(f"unknown out_dtype {out_dtype}")
    if made is None:
        return _empty(shape, dt, dev, stream)
    _need(made, (dt,), shape, name, dev)
    return made


def _cols(N, epilogue):
    if epilogue == MOE_EPI_SILU_MUL and N % 2:
        raise ValueError(f"SILU_MUL needs an even N (got {N})")
    return N // 2 if epilogue == MOE_EPI_SILU_MUL else N


def _groups(A, R, a_row_of, a_row_div, expert_offsets, E, dev):
    """Checks the description of the groups on the host's side (sizes; the contents stay on the device)."""
    _need(expert_offsets, _INT32, (E + 1,), "expert_offsets", dev)
    if a_row_of is None:
        if A.shape[0] < R:
            raise ValueError(f"A has {A.shape[0]} rows, the groups {R}")
    else:
        if a_row_of.dim() != 1 or a_row_of.shape[0] < R:
            raise ValueError(f"a_row_of must hold {R} indexes (got {tuple(a_row_of.shape)})")
        _need(a_row_of, _INT32, (...,), "a_row_of", dev)


def moe_i8_quantize(x, q=None, s=None, stream=None):
    """x bf16, fp16 or fp32 [rows, K] -> (codes int8 [rows, K], scales fp32 [rows])."""
    rows, K = _need(x, _ACT, (None, None), "x")
    dev = x.device
    if q is None:
        q = _empty((rows, K), torch.int8, dev, stream)
    else:
        _need(q, _I8, (rows, K), "q", dev)
    if s is None:
        s = _empty((rows,), torch.float32, dev, stream)
    else:
        _need(s, _F32, (rows,), "s", dev)
    _call(load().moe_i8_quantize, dev, stream, (q, s), x.data_ptr(), _IN[x.dtype], rows, K, q.data_ptr(), s.data_ptr())
    return q, s


def moe_gemm_i8(Aq, As, Wq, Ws, epilogue: int = MOE_EPI_NONE, out_dtype: int = MOE_OUT_BF16, C=None, stream=None):
    """Aq int8 [M, K], As fp32 [M], Wq int8 [N, K], Ws fp32 [N] -> C [M, N] ([M, N/2] for SILU_MUL)."""
    M, K = _need(Aq, _I8, (None, None), "Aq")
    dev = Aq.device
    _need(As, _F32, (M,), "As", dev)
    N, _ = _need(Wq, _I8, (None, K), "Wq", dev)
    _need(Ws, _F32, (N,), "Ws", dev)
    C = _out(C, (M, _cols(N, epilogue)), out_dtype, dev, "C", stream)
    _call(load().moe_gemm_i8, dev, stream, (C,), Aq.data_ptr(), As.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), M, N, K,
          epilogue, C.data_ptr(), out_dtype)
    return C


def moe_linear_i8_workspace_bytes(T: int, K: int) -> int:
    return int(load().moe_linear_i8_workspace_bytes(T, K))


def moe_linear_i8(x, Wq, Ws, epilogue: int = MOE_EPI_NONE, out_dtype: int = MOE_OUT_BF16, y=None, workspace=None,
                  stream=None):
    """x bf16, fp16 or fp32 [T, K], quantized on the fly, Wq int8 [N, K], Ws fp32 [N] -> y [T, N] ([T, N/2] for
    SILU_MUL)."""
    T, K = _need(x, _ACT, (None, None), "x")
    dev = x.device
    N, _ = _need(Wq, _I8, (None, K), "Wq", dev)
    _need(Ws, _F32, (N,), "Ws", dev)
    y = _out(y, (T, _cols(N, epilogue)), out_dtype, dev, "y", stream)
    lib, size = load(), 0
    if workspace is not None:
        size, = _need(workspace, _U8, (...,), "workspace", dev)
    else:
        size = lib.moe_linear_i8_workspace_bytes(T, K)
        if size:
            workspace = _empty((size,), torch.uint8, dev, stream, keep=False)
    _call(lib.moe_linear_i8, dev, stream, (y, workspace), x.data_ptr(), _IN[x.dtype], Wq.data_ptr(), Ws.data_ptr(), T, N, K,
          epilogue, y.data_ptr(), out_dtype, _ptr(workspace), size)
    return y


def moe_grouped_gemm_i8(Aq, As, a_row_of, a_row_div: int, Wq, Ws, expert_offsets, out_rows: int,
                        epilogue: int = MOE_EPI_NONE, out_dtype: int = MOE_OUT_BF16, C=None, stream=None):
    """Grouped int8 product over expert_offsets int32 [E + 1]: Aq int8 [*, K], As fp32 [*], Wq int8 [E, N, K],
    Ws fp32 [E, N] -> C [out_rows, N] ([out_rows, N/2] for SILU_MUL)."""
    rows, K = _need(Aq, _I8, (..., None), "Aq")
    dev = Aq.device
    _need(As, _F32, (rows,), "As", dev)
    E, N, _ = _need(Wq, _I8, (None, None, K), "Wq", dev)
    _need(Ws, _F32, (E, N), "Ws", dev)
    _groups(Aq, out_rows, a_row_of, a_row_div, expert_offsets, E, dev)
    C = _out(C, (out_rows, _cols(N, epilogue)), out_dtype, dev, "C", stream)
    _call(load().moe_grouped_gemm_i8, dev, stream, (C,), Aq.data_ptr(), As.data_ptr(), _ptr(a_row_of), a_row_div,
          Wq.data_ptr(), Ws.data_ptr(), expert_offsets.data_ptr(), out_rows, E, N, K, epilogue, C.data_ptr(), out_dtype)
    return C


def moe_ffn_i8_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_i8_workspace_bytes(T, H, I, E, k))


def _halves(N13, name):
    if N13 % 2:
        raise ValueError(f"{name} must hold as many gate as up rows (got {N13})")
    return N13 // 2


def _layer_io(x, router_logits, H, E, k, y, topk_ids_out, topk_w_out, workspace, need_bytes, stream):
    """Checks a layer's activations and optional buffers, makes y and the workspace where none is given."""
    dev, T = x.device, x.shape[0]
    _need(router_logits, _F32, (T, E), "router_logits", dev)
    if topk_ids_out is not None:
        _need(topk_ids_out, _INT32, (T, k), "topk_ids_out", dev)
    if topk_w_out is not None:
        _need(topk_w_out, _F32, (T, k), "topk_w_out", dev)
    y = _out(y, (T, H), MOE_OUT_BF16, dev, "y", stream)
    if workspace is None:
        workspace = _empty(max(need_bytes, 256), torch.uint8, dev, stream, keep=False)
    else:
        _need(workspace, _U8, (...,), "workspace", dev)
    return y, workspace


def moe_ffn_forward_i8(x, router_logits, w13_q, w13_s, w2_q, w2_s, k: int, y=None, topk_ids_out=None, topk_w_out=None,
                       workspace=None, stream=None):
    """Whole INT8 layer: x bf16 [T, H], logits fp32 [T, E], w13_q int8 [E, 2I, H] with scales fp32 [E, 2I], w2_q
    int8 [E, H, I] with scales fp32 [E, H] -> y bf16 [T, H]."""
    T, H = _need(x, (torch.bfloat16,), (None, None), "x")
    dev = x.device
    E, N13, _ = _need(w13_q, _I8, (None, None, H), "w13_q", dev)
    I = _halves(N13, "w13_q")
    _need(w13_s, _F32, (E, 2 * I), "w13_s", dev)
    _need(w2_q, _I8, (E, H, I), "w2_q", dev)
    _need(w2_s, _F32, (E, H), "w2_s", dev)
    y, workspace = _layer_io(x, router_logits, H, E, k, y, topk_ids_out, topk_w_out, workspace,
                             moe_ffn_i8_workspace_bytes(T, H, I, E, k), stream)
    _call(load().moe_ffn_forward_i8, dev, stream, (y, workspace), x.data_ptr(), router_logits.data_ptr(), T, H, I, E, k,
          w13_q.data_ptr(), w13_s.data_ptr(), w2_q.data_ptr(), w2_s.data_ptr(), y.data_ptr(), _ptr(topk_ids_out),
          _ptr(topk_w_out), workspace.data_ptr(), workspace.numel())
    return y


def moe_grouped_gemm_w16(A, a_row_of, a_row_div: int, W, expert_offsets, out_rows: int, epilogue: int = MOE_EPI_NONE,
                         out_dtype: int = None, C=None, stream=None):
    """Grouped product over expert_offsets int32 [E + 1]: A [*, K] and W [E, N, K], both bf16 or both fp16 -> C
    [out_rows, N] ([out_rows, N/2] for SILU_MUL) of out_dtype (default: the operands' type)."""
    _, K = _need(A, _W16, (..., None), "A")
    dev, dt = A.device, A.dtype
    E, N, _ = _need(W, (dt,), (None, None, K), "W", dev)
    _groups(A, out_rows, a_row_of, a_row_div, expert_offsets, E, dev)
    out_dtype = _OUT[dt] if out_dtype is None else out_dtype
    C = _out(C, (out_rows, _cols(N, epilogue)), out_dtype, dev, "C", stream)
    _call(load().moe_grouped_gemm_w16, dev, stream, (C,), A.data_ptr(), _ptr(a_row_of), a_row_div, W.data_ptr(), _IN[dt],
          expert_offsets.data_ptr(), out_rows, E, N, K, epilogue, C.data_ptr(), out_dtype)
    return C


def moe_grouped_gemm_w16_dx(dC, W, expert_offsets, out_dtype: int = None, dA=None, stream=None):
    """Row gradients of moe_grouped_gemm_w16: dC [R, N] and W [E, N, K] of one type -> dA [R, K] of out_dtype
    (default: the operands' type)."""
    R, N = _need(dC, _W16, (None, None), "dC")
    dev, dt = dC.device, dC.dtype
    E, _, K = _need(W, (dt,), (None, N, None), "W", dev)
    _need(expert_offsets, _INT32, (E + 1,), "expert_offsets", dev)
    out_dtype = _OUT[dt] if out_dtype is None else out_dtype
    dA = _out(dA, (R, K), out_dtype, dev, "dA", stream)
    _call(load().moe_grouped_gemm_w16_dx, dev, stream, (dA,), dC.data_ptr(), W.data_ptr(), _IN[dt],
          expert_offsets.data_ptr(), R, E, N, K, dA.data_ptr(), out_dtype)
    return dA


def moe_grouped_gemm_w16_dw_workspace_bytes(R: int, E: int, N: int, K: int) -> int:
    return int(load().moe_grouped_gemm_w16_dw_workspace_bytes(R, E, N, K))


def moe_grouped_gemm_w16_dw(dC, A, a_row_of, a_row_div: int, expert_offsets, out_dtype: int = None, dW=None,
                            workspace=None, stream=None):
    """Weight gradients of moe_grouped_gemm_w16: dC [R, N] and A [*, K] of one type -> dW [E, N, K] of out_dtype
    (default: the operands' type); zeros for experts without rows."""
    R, N = _need(dC, _W16, (None, None), "dC")
    dev, dt = dC.device, dC.dtype
    _, K = _need(A, (dt,), (..., None), "A", dev)
    if expert_offsets.dim() != 1 or expert_offsets.shape[0] < 2:
        raise ValueError(f"expert_offsets must have the shape (E + 1,) (got {tuple(expert_offsets.shape)})")
    E = expert_offsets.shape[0] - 1
    _groups(A, R, a_row_of, a_row_div, expert_offsets, E, dev)
    out_dtype = _OUT[dt] if out_dtype is None else out_dtype
    dW = _out(dW, (E, N, K), out_dtype, dev, "dW", stream)
    lib, size = load(), 0
    if workspace is not None:
        size, = _need(workspace, _U8, (...,), "workspace", dev)
    else:
        size = lib.moe_grouped_gemm_w16_dw_workspace_bytes(R, E, N, K)
        if size:
            workspace = _empty((size,), torch.uint8, dev, stream, keep=False)
    _call(lib.moe_grouped_gemm_w16_dw, dev, stream, (dW, workspace), dC.data_ptr(), A.data_ptr(), _ptr(a_row_of), a_row_div,
          _IN[dt], expert_offsets.data_ptr(), R, E, N, K, dW.data_ptr(), out_dtype, _ptr(workspace), size)
    return dW


def _silu_shape(G):
    R, C = _need(G, _W16, (None, None), "G")
    if C % 2:
        raise ValueError(f"G must have an even number of columns (got {C})")
    return R, C // 2


def moe_silu_mul(G, h=None, stream=None):
    """G [R, 2I] (gate, up) bf16 or fp16 -> h = silu(gate) * up [R, I] of its type."""
    R, I = _silu_shape(G)
    h = _out(h, (R, I), _OUT[G.dtype], G.device, "h", stream)
    _call(load().moe_silu_mul, G.device, stream, (h,), G.data_ptr(), _IN[G.dtype], R, I, h.data_ptr())
    return h


def moe_silu_mul_grad(G, dh, dG=None, stream=None):
    """Gradient of moe_silu_mul: G [R, 2I], dh [R, I] -> dG [R, 2I]."""
    R, I = _silu_shape(G)
    _need(dh, (G.dtype,), (R, I), "dh", G.device)
    dG = _out(dG, (R, 2 * I), _OUT[G.dtype], G.device, "dG", stream)
    _call(load().moe_silu_mul_grad, G.device, stream, (dG,), G.data_ptr(), dh.data_ptr(), _IN[G.dtype], R, I, dG.data_ptr())
    return dG


def moe_ffn_w16_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_w16_workspace_bytes(T, H, I, E, k))


def moe_ffn_forward_w16(x, router_logits, w13, w2, k: int, y=None, topk_ids_out=None, topk_w_out=None, workspace=None,
                        stream=None):
    """Whole layer with bf16 weights: x bf16 [T, H], logits fp32 [T, E], w13 bf16 [E, 2I, H], w2 bf16 [E, H, I] -> y
    bf16 [T, H]."""
    bf16 = (torch.bfloat16,)
    T, H = _need(x, bf16, (None, None), "x")
    dev = x.device
    E, N13, _ = _need(w13, bf16, (None, None, H), "w13", dev)
    I = _halves(N13, "w13")
    _need(w2, bf16, (E, H, I), "w2", dev)
    y, workspace = _layer_io(x, router_logits, H, E, k, y, topk_ids_out, topk_w_out, workspace,
                             moe_ffn_w16_workspace_bytes(T, H, I, E, k), stream)
    _call(load().moe_ffn_forward_w16, dev, stream, (y, workspace), x.data_ptr(), router_logits.data_ptr(), T, H, I, E, k,
          w13.data_ptr(), w2.data_ptr(), y.data_ptr(), _ptr(topk_ids_out), _ptr(topk_w_out), workspace.data_ptr(),
          workspace.numel())
    return y


def _made_like(made, x, dtype, name, stream):
    """The caller's tensor of x's shape, checked, or a new one."""
    if made is not None:
        _need(made, (dtype,), tuple(x.shape), name, x.device)
        return made
    return _empty(x.shape, dtype, x.device, stream, like=x)


def moe_rmsnorm_add(x, weight, eps: float, residual=None, quant: int = MOE_QUANT_NONE, want_y: bool = True, s=None, y=None,
                    q=None, q_scale=None, stream=None):
    """x [T, H] bf16 or fp16, weight [H] of its type or fp32, residual [T, H] or None -> (s, y, q, q_scale): s = x +
    residual (None without one), y the normalised rows (None where want_y is false and no y is given), q the codes [T, H]
    (int8, or E4M3 bytes in uint8) and q_scale fp32 [T] or [T, H / 128] (None for MOE_QUANT_NONE)."""
    T, H = _need(x, _W16, (None, None), "x")
    dev, dt = x.device, x.dtype
    _need(weight, (dt, torch.float32), (H,), "weight", dev)
    if residual is not None:
        _need(residual, (dt,), (T, H), "residual", dev)
        s = _made_like(s, x, dt, "s", stream)
    elif s is not None:
        raise ValueError("s is the sum with a residual, and none is given")
    if want_y or y is not None:
        y = _made_like(y, x, dt, "y", stream)
    if quant == MOE_QUANT_NONE:
        if q is not None or q_scale is not None:
            raise ValueError("q and q_scale belong to a quant of MOE_QUANT_I8 or MOE_QUANT_F8")
    elif quant == MOE_QUANT_I8 or quant == MOE_QUANT_F8:
        if quant == MOE_QUANT_F8 and H % 128:
            raise ValueError(f"MOE_QUANT_F8 needs a multiple of 128 columns (got {H})")
        q = _made_like(q, x, torch.int8 if quant == MOE_QUANT_I8 else torch.uint8, "q", stream)
        q_scale = _out(q_scale, (T,) if quant == MOE_QUANT_I8 else (T, H // 128), MOE_OUT_F32, dev, "q_scale", stream)
    else:
        raise ValueError(f"unknown quant {quant}")
    _call(load().moe_rmsnorm_add, dev, stream, (s, y, q, q_scale), x.data_ptr(), _ptr(residual), _IN[dt], weight.data_ptr(),
          _IN[weight.dtype], eps, T, H, _ptr(s), _ptr(y), quant, _ptr(q), _ptr(q_scale))
    return s, y, q, q_scale


def moe_rmsnorm_add_grad_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_rmsnorm_add_grad_workspace_bytes(T, H))


def moe_rmsnorm_add_grad(dy, s, weight, eps: float, ds=None, out_dtype: int = None, dx=None, dweight=None, workspace=None,
                         stream=None):
    """Gradient of moe_rmsnorm_add: dy [T, H], s [T, H] (the forward pass's sum, or its x), ds [T, H] or None -> (dx [T, H],
    of x and of the residual, dweight [H] of out_dtype, by default the weight's type)."""
    T, H = _need(s, _W16, (None, None), "s")
    dev, dt = s.device, s.dtype
    _need(dy, (dt,), (T, H), "dy", dev)
    _need(weight, (dt, torch.float32), (H,), "weight", dev)
    if ds is not None:
        _need(ds, (dt,), (T, H), "ds", dev)
    out_dtype = _OUT[weight.dtype] if out_dtype is None else out_dtype
    dx = _made_like(dx, s, dt, "dx", stream)
    dweight = _out(dweight, (H,), out_dtype, dev, "dweight", stream)
    lib, size = load(), 0
    if workspace is not None:
        size, = _need(workspace, _U8, (...,), "workspace", dev)
    else:
        size = lib.moe_rmsnorm_add_grad_workspace_bytes(T, H)
        if size:
            workspace = _empty((size,), torch.uint8, dev, stream, keep=False)
    _call(lib.moe_rmsnorm_add_grad, dev, stream, (dx, dweight, workspace), dy.data_ptr(), s.data_ptr(), _IN[dt],
          weight.data_ptr(), _IN[weight.dtype], eps, _ptr(ds), T, H, dx.data_ptr(), dweight.data_ptr(), out_dtype,
          _ptr(workspace), size)
    return dx, dweight


def moe_ffn_few_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load().moe_ffn_few_workspace_bytes(T, H, I, E, k))


def moe_ffn_few_w16(x, router_logits, w13, w2, k: int, y=None, topk_ids_out=None, topk_w_out=None, workspace=None,
                    stream=None):
    """Whole layer for at most 16 tokens in two launches, bf16 weights (arguments of moe_ffn_forward_w16)."""
    T, H = _need(x, _BF16, (None, None), "x")
    dev = x.device
    E, N13, _ = _need(w13, _BF16, (None, None, H), "w13", dev)
    I = _halves(N13, "w13")
    _need(w2, _BF16, (E, H, I), "w2", dev)
    lib = load()
    y, workspace = _layer_io(x, router_logits, H, E, k, y, topk_ids_out, topk_w_out, workspace,
                             lib.moe_ffn_few_workspace_bytes(T, H, I, E, k), stream)
    _call(lib.moe_ffn_few_w16, dev, stream, (y, topk_ids_out, topk_w_out, workspace), x.data_ptr(), router_logits.data_ptr(), T,
          H, I, E, k, w13.data_ptr(), w2.data_ptr(), y.data_ptr(), _ptr(topk_ids_out), _ptr(topk_w_out), workspace.data_ptr(),
          workspace.numel())
    return y


def moe_ffn_few_w8a16(x, router_logits, w13_q, w13_s, w2_q, w2_s, k: int, y=None, topk_ids_out=None, topk_w_out=None,
                      workspace=None, stream=None):
    """Whole layer for at most 16 tokens in two launches, int8 weights with channel scales (arguments of
    moe_ffn_forward_i8), activations not quantized."""
    T, H = _need(x, _BF16, (None, None), "x")
    dev = x.device
    E, N13, _ = _need(w13_q, _I8, (None, None, H), "w13_q", dev)
    I = _halves(N13, "w13_q")
    _need(w13_s, _F32, (E, 2 * I), "w13_s", dev)
    _need(w2_q, _I8, (E, H, I), "w2_q", dev)
    _need(w2_s, _F32, (E, H), "w2_s", dev)
    lib = load()
    y, workspace = _layer_io(x, router_logits, H, E, k, y, topk_ids_out, topk_w_out, workspace,
                             lib.moe_ffn_few_workspace_bytes(T, H, I, E, k), stream)
    _call(lib.moe_ffn_few_w8a16, dev, stream, (y, topk_ids_out, topk_w_out, workspace), x.data_ptr(), router_logits.data_ptr(),
          T, H, I, E, k, w13_q.data_ptr(), w13_s.data_ptr(), w2_q.data_ptr(), w2_s.data_ptr(), y.data_ptr(),
          _ptr(topk_ids_out), _ptr(topk_w_out), workspace.data_ptr(), workspace.numel())
    return y
