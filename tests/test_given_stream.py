"""Calls on a given stream (stream=): the tensors that a wrapper makes for one belong to that stream.  A block that
the current stream's allocator hands out may still be in use by work queued on the current stream, and the given one
does not wait for it."""
import ast
import inspect

import pytest
import torch

import moe_w4a16_grouped_amd as moe
from moe_w4a16_grouped_amd import _lib

BF16, F32 = torch.bfloat16, torch.float32


def test_tensors_are_made_in_one_place():
    """Every tensor of the binding comes from _empty with the call's stream."""
    makers = {"empty", "empty_like", "zeros", "zeros_like", "ones", "full", "new_empty"}
    for node in ast.walk(ast.parse(inspect.getsource(_lib))):
        if not isinstance(node, ast.FunctionDef):
            continue
        for call in (n for n in ast.walk(node) if isinstance(n, ast.Call)):
            if isinstance(call.func, ast.Attribute) and call.func.attr in makers:
                assert node.name == "_empty", (node.name, ast.unparse(call))
            if isinstance(call.func, ast.Name) and call.func.id in ("_empty", "_out", "_layer_io"):
                assert any(isinstance(a, ast.Name) and a.id == "stream" for a in call.args), (node.name, ast.unparse(call))


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _calls():
    """name -> (call of stream, bytes of its workspace)."""
    R, N, K, E, k = 4096, 1024, 512, 4, 2
    x, W, logits = _rand((R, K), BF16, 1), _rand((E, N, K), BF16, 2, K ** -0.5), _rand((R, E), F32, 3)
    off = torch.tensor([0, 1000, 1000, 3000, R], dtype=torch.int32, device="cuda")
    dC, G = _rand((R, N), BF16, 4), _rand((R, 2 * N), BF16, 5)
    wq, ws = moe.moe_i8_quantize(W.view(-1, K))
    w2 = _rand((E, K, N // 2), BF16, 6, 0.05)
    ids, w = moe.moe_route_topk(logits, k)
    al = moe.moe_align(ids, E, 64)
    O = _rand((R * k, K), F32, 7)
    return {
        "i8_quantize": (lambda s: moe.moe_i8_quantize(x, stream=s), 0),
        "linear_i8": (lambda s: moe.moe_linear_i8(x, wq[:N], ws[:N], stream=s), moe.moe_linear_i8_workspace_bytes(R, K)),
        "w16": (lambda s: moe.moe_grouped_gemm_w16(x, None, 1, W, off, R, stream=s), 0),
        "w16_dx": (lambda s: moe.moe_grouped_gemm_w16_dx(dC, W, off, stream=s), 0),
        "w16_dw": (lambda s: moe.moe_grouped_gemm_w16_dw(dC, x, None, 1, off, stream=s),
                   moe.moe_grouped_gemm_w16_dw_workspace_bytes(R, E, N, K)),
        "silu_mul": (lambda s: moe.moe_silu_mul(G, stream=s), 0),
        "ffn_w16": (lambda s: moe.moe_ffn_forward_w16(x, logits, W, w2, k, stream=s), moe.moe_ffn_w16_workspace_bytes(R, K, N // 2, E, k)),
        "route": (lambda s: moe.moe_route_topk(logits, k, stream=s), 0),
        "combine": (lambda s: moe.moe_combine(O, al["inv_perm"], w, stream=s), 0),
        "mx_quantize": (lambda s: moe.moe_mx_quantize(x, stream=s), 0),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["i8_quantize", "linear_i8", "w16", "w16_dx", "w16_dw", "silu_mul", "ffn_w16", "route", "combine",
                                  "mx_quantize"])
def test_blocks_in_use_on_the_current_stream_are_left_alone(name):
    """Blocks of the call's sizes are freed while work queued on the current stream has still to read them; the
    call on the other stream waits for nothing, as its inputs are ready."""
    call, workspace = _calls()[name]
    listed = lambda out: list(out) if isinstance(out, tuple) else [out]
    want = [t.clone() for t in listed(call(None))]
    busy, other = _rand((4096, 4096), F32, 8), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [t.numel() * t.element_size() for t in want] + ([workspace] if workspace else [])
    victims = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 2.0 ** -12
    read = [v.clone() for v in victims]
    del victims
    got = listed(call(other))
    torch.cuda.synchronize()
    assert all(bool((r == 7).all()) for r in read)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_results_may_be_freed_on_the_current_stream():
    """A result of the other stream, read by queued work on the current one and freed: the other stream's next
    call does not write over it before it is read."""
    G, other = _rand((4096, 2048), BF16, 1), torch.cuda.Stream()
    G2, want = -G, moe.moe_silu_mul(G)
    busy = _rand((4096, 4096), F32, 8)
    torch.cuda.synchronize()
    h = moe.moe_silu_mul(G, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    for _ in range(20):
        busy = busy @ busy * 2.0 ** -12
    read = h.clone()
    del h
    later = moe.moe_silu_mul(G2, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(read, want) and torch.equal(later, moe.moe_silu_mul(G2))


@pytest.mark.gpu
def test_a_given_stream_within_a_captured_graph():
    """Two streams of one captured graph, with tensors made on both; replayed with other inputs, eager calls between."""
    x, W = _rand((640, 256), BF16, 1), _rand((2, 512, 256), BF16, 2, 0.06)
    off = torch.tensor([0, 300, 640], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def both(a, s):
        here = torch.cuda.current_stream()
        if s is not None:
            s.wait_stream(here)
        G = moe.moe_grouped_gemm_w16(a, None, 1, W, off, 640, stream=s)
        q = moe.moe_i8_quantize(a)
        h = moe.moe_silu_mul(G, stream=s)
        if s is not None:
            here.wait_stream(s)
        return [G, *q, h, moe.moe_silu_mul_grad(G, h)]

    live = x.clone()
    both(live, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(live, side)
    for seed in (3, 4, 3):
        src = _rand((640, 256), BF16, seed)
        live.copy_(src)
        graph.replay()
        want = both(src, None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed
