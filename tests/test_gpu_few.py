"""The layer for a few tokens in two launches (bf16 weights, int8 weights) against the layer in 64 bits.

Bounds.  G: fp32 sums of K products (ragged_util.sum_bound), for int8 the scale's product.  h: ragged_util.silu_bound, and the two
bf16 parts (what the first leaves is at most 2^-8 of h, rounded by at most half a step of 2^-8 more: 2^-16).  O: the
products' sums with h's error, over both parts of h.  y: the weights of the slots (fp32 exponentials and a quotient:
2^-20), k rounded multiply-adds, and half a step of bf16."""
import pytest
import torch

import moe_w4a16_grouped_amd as moe
from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


class Layer:
    def __init__(self, T, E, k, H, I, int8, seed=0, logits=None):
        self.k, self.int8 = k, int8
        self.x = _rand((T, H), BF16, seed)
        self.logits = _rand((T, E), F32, seed + 1) if logits is None else logits
        if int8:
            self.w13, self.w13_s = (t.view(E, 2 * I, -1).squeeze(-1) for t in moe.moe_i8_quantize(_rand((E * 2 * I, H), F32, seed + 2, H ** -0.5)))
            self.w2, self.w2_s = (t.view(E, H, -1).squeeze(-1) for t in moe.moe_i8_quantize(_rand((E * H, I), F32, seed + 3, I ** -0.5)))
        else:
            self.w13, self.w2 = _rand((E, 2 * I, H), BF16, seed + 2, H ** -0.5), _rand((E, H, I), BF16, seed + 3, I ** -0.5)

    def run(self, **more):
        if self.int8:
            return moe.moe_ffn_few_w8a16(self.x, self.logits, self.w13, self.w13_s, self.w2, self.w2_s, self.k, **more)
        return moe.moe_ffn_few_w16(self.x, self.logits, self.w13, self.w2, self.k, **more)

    def routing(self):
        top, ids = torch.sort(self.logits, dim=1, descending=True, stable=True)
        return ids[:, :self.k], torch.softmax(top[:, :self.k].double(), dim=1)

    def reference(self):
        """(y, bound before y's own rounding) in 64 bits."""
        ids, weight = self.routing()
        T, H = self.x.shape
        I = self.w2.shape[2]
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        err, mass = torch.zeros_like(y), torch.zeros_like(y)
        for e in torch.unique(ids).tolist():
            t, slot = torch.nonzero(ids == e, as_tuple=True)
            up, down, scaled = self.w13[e].double(), self.w2[e].double(), 0.0
            if self.int8:
                up, down, scaled = up * self.w13_s[e].double()[:, None], down * self.w2_s[e].double()[:, None], U
            x = self.x[t].double()
            G, G_mass = x @ up.t(), x.abs() @ up.abs().t()
            G_err = ru.sum_bound(H, G_mass) + scaled * G.abs()
            h, h_err = ru.silu_mul(G), ru.silu_bound(G, G_err)
            h_err = h_err + 2.0 ** -16 * (h.abs() + h_err)
            O, O_mass = h @ down.t(), (h.abs() + h_err) @ down.abs().t()
            O_err = h_err @ down.abs().t() + ru.sum_bound(2 * I, 1.01 * O_mass) + scaled * O.abs()
            w = weight[t, slot][:, None]
            y.index_add_(0, t, w * O)
            err.index_add_(0, t, w * (O_err + 2.0 ** -20 * O.abs()))
            mass.index_add_(0, t, w * O.abs())
        return y, err + (self.k + 1) * U * mass

    def check(self, y, label=""):
        ref, err = self.reference()
        ru.assert_close(y, ref, err, label)


SHAPES = [  # T, E, k, H, I
    (1, 128, 8, 2048, 768), (2, 4, 1, 16, 16), (3, 8, 2, 48, 32), (7, 60, 6, 1040, 336), (8, 128, 8, 512, 256), (9, 16, 3, 272, 80),
    (16, 256, 8, 1024, 512), (16, 8, 2, 4096, 1024), (5, 300, 10, 256, 64), (13, 1024, 16, 64, 48), (16, 16, 16, 128, 112),
    (11, 5, 5, 2064, 1040), (4, 2, 1, 528, 4000), (16, 4, 2, 8192, 64), (3, 4, 3, 32768, 16), (1, 1, 1, 65536, 32),
]


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
def test_few(T, E, k, H, I, int8):
    L = Layer(T, E, k, H, I, int8, seed=T + E)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    y = torch.full((T, H), float("nan"), dtype=BF16, device="cuda")
    ws = torch.full((moe.moe_ffn_few_workspace_bytes(T, H, I, E, k),), 0xFF, dtype=torch.uint8, device="cuda")
    assert L.run(y=y, topk_ids_out=ids, topk_w_out=w, workspace=ws) is y
    want_ids, want_w = moe.moe_route_topk(L.logits, k)
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
    assert torch.equal(ids.long(), L.routing()[0])
    L.check(y)
    assert torch.equal(L.run(), y)  # the same bits, without the optional buffers


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
def test_crowded_and_tied(int8):
    """All tokens on the same experts (more than eight to one), and equal logits in the order of their experts."""
    T, E, k, H, I = 16, 24, 4, 256, 96
    row = _rand((1, E), F32, 3)
    for logits in (row.repeat(T, 1), torch.zeros((T, E), device="cuda"), torch.where(torch.arange(E, device="cuda") % 5 == 0, 2.0, -0.0).repeat(T, 1)):
        L = Layer(T, E, k, H, I, int8, seed=4, logits=logits.contiguous())
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        L.check(L.run(topk_ids_out=ids))
        assert torch.equal(ids.long(), L.routing()[0])
    hot = _rand((T, E), F32, 5)
    hot[:9, 7] += 20  # nine of sixteen tokens
    L = Layer(T, E, k, H, I, int8, seed=6, logits=hot)
    L.check(L.run())


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
@pytest.mark.parametrize("lowest", [-3.4028234663852886e38, float("-inf")])
def test_masked_experts(int8, lowest):
    """Experts that a mask closes get the weight 0 where fewer than k are left open, and never reach y, whatever they hold."""
    T, E, k, H, I = 6, 16, 4, 128, 64
    logits = _rand((T, E), F32, 1)
    logits[:, 2:] = lowest
    L = Layer(T, E, k, H, I, int8, seed=2, logits=logits)
    w = torch.empty((T, k), device="cuda")
    y = L.run(topk_w_out=w)
    assert not bool(w[:, 2:].any())
    L.check(y)
    if int8:
        L.w13_s[2:], L.w2_s[2:] = float("nan"), float("inf")
    else:
        L.w13[2:], L.w2[2:] = float("nan"), float("inf")
    assert torch.equal(L.run(), y)


def test_values_without_end_stay_with_their_token():
    """An infinity or NaN in one token, or in an expert that one token chose, reaches that token alone."""
    T, E, k, H, I = 8, 32, 2, 128, 64
    L = Layer(T, E, k, H, I, False, seed=9)
    plain = L.run()
    L.x[2, 5], L.x[5, 7] = float("nan"), float("inf")
    y = L.run()
    rest = torch.tensor([0, 1, 3, 4, 6, 7], device="cuda")
    assert torch.equal(y[rest], plain[rest]) and bool(y[2].isnan().all())
    L = Layer(T, E, k, H, I, False, seed=9)
    ids = L.routing()[0]
    e = int(ids[0, 0])
    L.w13[e] = float("nan")
    y = L.run()
    hit = (ids == e).any(dim=1)
    assert torch.equal(y[~hit], plain[~hit]) and bool(y[hit].isnan().all())
    idle = [e for e in range(E) if not bool((ids == e).any())]
    L = Layer(T, E, k, H, I, False, seed=9)
    L.w13[idle], L.w2[idle] = float("nan"), float("nan")
    assert torch.equal(L.run(), plain)


def test_large_activations():
    """h beyond fp16's range and tiny ones, of both signs."""
    for scale in (1e4, 1e-6):
        L = Layer(4, 8, 2, 256, 128, False, seed=3)
        L.x = (L.x.float() * scale).to(BF16)
        L.w2 = (L.w2.float() * 1e-3).to(BF16)
        L.check(L.run())


def test_weights_past_four_gib():
    """Offsets of experts and rows beyond 2^32 bytes."""
    T, E, k, H, I = 2, 18, 2, 4096, 16384
    logits = torch.full((T, E), -5.0, device="cuda")
    logits[0, 17], logits[0, 16], logits[1, 17], logits[1, 0] = 3.0, 2.0, 1.0, 0.5
    L = Layer(T, 2, 2, H, I, False, seed=5)
    w13, w2 = L.w13, L.w2
    L.w13 = torch.zeros((E, 2 * I, H), dtype=BF16, device="cuda")
    L.w2 = torch.zeros((E, H, I), dtype=BF16, device="cuda")
    L.w13[16:], L.w2[16:], L.logits = w13, w2, logits
    L.check(L.run())


def test_rows_behind_and_no_tokens():
    L = Layer(3, 8, 2, 128, 64, False)
    y = torch.full((5, 128), 7.0, dtype=BF16, device="cuda")
    L.run(y=y[:3])
    assert bool((y[3:] == 7.0).all())
    L.x, L.logits = L.x[:0], L.logits[:0]
    assert L.run().shape == (0, 128)


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
def test_stream_and_graph(int8):
    L = Layer(10, 64, 6, 512, 192, int8, seed=1)
    ref = L.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = L.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.run()
    for seed in range(4):
        L.x.copy_(_rand(tuple(L.x.shape), BF16, 30 + seed))
        L.logits.copy_(_rand(tuple(L.logits.shape), F32, 40 + seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, L.run())


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 16, 4, 512, 1024), (1, 300, 16, 528, 1040), (1, 9, 2, 32, 4112), (2, 40, 7, 1280, 544), (16, 5, 3, 4112, 48),
                                       (15, 31, 1, 768, 528), (4, 1024, 3, 144, 16), (3, 9, 2, 1040, 272), (5, 40, 3, 2064, 288), (6, 40, 3, 3344, 96),
                                       (1, 9, 3, 2080, 272), (1, 9, 3, 4112, 96), (9, 6, 4, 2576, 272), (3, 30, 3, 7168, 64), (1, 9, 3, 1296, 48)])
def test_mixes_of_the_rules(T, E, k, H, I, int8):
    """Short rows and narrow outputs, single tokens, crowded experts, in the mixes that SHAPES leaves out."""
    L = Layer(T, E, k, H, I, int8, seed=T * E)
    L.check(L.run())


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
@pytest.mark.parametrize("T,E,k,H,I", [(11, 60, 8, 224, 2064), (1, 20, 10, 240, 10256), (14, 4, 4, 160, 5024), (16, 64, 16, 1024, 1552), (2, 150, 16, 16, 8208)])
def test_groups_of_the_second_launch(T, E, k, H, I, int8):
    """Few columns and a long contraction: workgroups share the columns' units, and a third launch adds their parts."""
    L = Layer(T, E, k, H, I, int8, seed=T + k)
    ws = torch.full((moe.moe_ffn_few_workspace_bytes(T, H, I, E, k),), 0xFF, dtype=torch.uint8, device="cuda")
    y = L.run(workspace=ws)
    L.check(y)
    assert torch.equal(L.run(workspace=ws), y)
    L.logits[:, 0] = float("-inf")  # a closed expert holds anything (where E is k it is chosen, with weight 0: 0 * NaN in the reference)
    y = L.run()
    L.check(y)
    L.w2.view(torch.uint8 if int8 else torch.int16)[0] = 0x7F if int8 else 0x7FC0
    assert torch.equal(L.run(), y)


def test_scales_on_four_bytes():
    """Scales need four bytes of alignment only."""
    for T, E, k, H, I in ((12, 20, 4, 256, 112), (1, 20, 4, 2048, 64), (1, 20, 4, 256, 640)):
        L = Layer(T, E, k, H, I, True, seed=3)
        y = L.run()
        for name in ("w13_s", "w2_s"):
            t = getattr(L, name)
            moved = torch.full((t.numel() + 4,), float("nan"), device="cuda")
            moved[1:-3] = t.view(-1)
            setattr(L, name, moved[1:-3].view(t.shape))
        assert torch.equal(L.run(), y)


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
def test_two_graphs_of_one_workspace(int8):
    """A token group a launch, captured: 5 tokens of 16384 columns are groups of 4 and 1.  Two graphs share a workspace."""
    layers = [Layer(5, 6, 2, 16384, 64, int8, seed=1), Layer(16, 30, 5, 512, 272, int8, seed=2)]
    size = max(moe.moe_ffn_few_workspace_bytes(*L.x.shape, L.w2.shape[2], L.logits.shape[1], L.k) for L in layers)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    for L in layers:
        L.check(L.run(workspace=ws))
    graphs, outs = [], []
    for L in layers:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(L.run(workspace=ws))
    for seed in range(4):
        for L in layers:
            L.x.copy_(_rand(tuple(L.x.shape), BF16, 50 + seed))
            L.logits.copy_(_rand(tuple(L.logits.shape), F32, 60 + seed))
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for L, out in zip(layers, outs):
            assert torch.equal(out, L.run())


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    layers = [Layer(16, 64, 6, 1024, 512, False, seed=1), Layer(9, 40, 4, 2048, 256, True, seed=2)]
    want = [L.run() for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[L.run(stream=s) for L, s in zip(layers, streams)] for _ in range(8)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_close_to_the_layers_of_any_size():
    """The layer that these launches stand in for rounds h to bf16 (2^-8 of it, half a step), and y the same."""
    for int8 in (False, True):
        L = Layer(6, 32, 4, 512, 256, int8, seed=8)
        y = L.run().double()
        if int8:
            other = moe.moe_ffn_forward_i8(L.x, L.logits, L.w13, L.w13_s, L.w2, L.w2_s, L.k).double()
        else:
            other = moe.moe_ffn_forward_w16(L.x, L.logits, L.w13, L.w2, L.k).double()
        assert float((y - other).norm() / other.norm()) < (0.03 if int8 else 0.01)


def test_decode_step():
    """norm with the residual -> router -> layer for a few tokens -> next norm, each against the 64-bit form of its inputs."""
    T, E, k, H, I = 5, 32, 4, 512, 256
    L = Layer(T, E, k, H, I, True, seed=12)
    res, weight, w_router = _rand((T, H), BF16, 1), (_rand((H,), F32, 2) * 0.1 + 1), _rand((E, H), BF16, 3, H ** -0.5)
    s, y, _, _ = moe.moe_rmsnorm_add(L.x, weight, 1e-6, residual=res)
    L.x, L.logits = y, moe.moe_router_logits(y, w_router)
    out = L.run()
    L.check(out)
    s2, y2, q2, scale2 = moe.moe_rmsnorm_add(out, weight, 1e-6, residual=s, quant=moe.MOE_QUANT_I8)
    total = (out.float() + s.float()).to(BF16)
    assert torch.equal(s2, total)
    v = total.double()
    want = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + 1e-6) * weight.double()
    ru.assert_close(y2, want, 4.6 * U * want.abs())  # (see test_gpu_norm)
    assert bool(((q2.double() * scale2.double()[:, None] - want).abs() <= scale2.double()[:, None] * 0.5001).all())


def test_refusals_of_the_binding():
    L = Layer(4, 8, 2, 64, 32, False)
    bad = [lambda: moe.moe_ffn_few_w16(L.x.half(), L.logits, L.w13, L.w2, 2), lambda: moe.moe_ffn_few_w16(L.x, L.logits[:2], L.w13, L.w2, 2),
           lambda: moe.moe_ffn_few_w16(L.x, L.logits, L.w13, L.w2.transpose(1, 2), 2), lambda: moe.moe_ffn_few_w16(L.x, L.logits, L.w13[:, :63], L.w2, 2),
           lambda: L.run(topk_ids_out=torch.zeros((4, 2), dtype=torch.int64, device="cuda")),
           lambda: L.run(topk_w_out=torch.zeros((4, 3), device="cuda")), lambda: L.run(y=torch.zeros((3, 64), dtype=BF16, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoEError):
        L.run(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoEError):
        moe.moe_ffn_few_w16(L.x, L.logits, L.w13, L.w2, 9)
    with pytest.raises(moe.MoEError):
        moe.moe_ffn_few_w16(L.x.repeat(5, 1), L.logits.repeat(5, 1), L.w13, L.w2, 2)


def _table(ws, T, k, I):
    """The entries that the first launch leaves in the workspace, behind h: (expert, rows) in the order in which the second takes them."""
    at = (T * k * I * 4 + 255) // 256 * 256
    ints = ws[at:at + 32 * (1 + T * k)].view(torch.int32).view(-1, 8).cpu()
    rows = ints[1:, 2:6].contiguous().view(torch.int16)
    return [(int(e[0]), rows[i, :int(e[1])].tolist()) for i, e in enumerate(ints[1:1 + int(ints[0, 0])])]


@pytest.mark.parametrize("int8", [False, True], ids=["w16", "w8a16"])
@pytest.mark.parametrize("T,E,k,H,I", [(16, 128, 16, 1024, 1024), (16, 300, 16, 528, 2064), (15, 100, 16, 1024, 2064), (16, 80, 16, 272, 4112),
                                       (3, 8, 2, 48, 32), (1, 20, 10, 240, 1040)])
def test_entries_stand_in_a_fixed_order(T, E, k, H, I, int8):
    """Experts ascending (of one token: by slot) with their first rows, then in the same order what is left of those with more rows than an entry takes.
    Where workgroups share columns a place in this table decides with which others an entry is summed, so arrival order must
    not enter it.  The larger cases have such experts on both sides of the 64th: their entries come from two waves."""
    logits = _rand((T, E), F32, 1)
    if E >= 80:
        logits[:, [3, 40, E - 2]] += 20.0  # all tokens on these
    L = Layer(T, E, k, H, I, int8, seed=T + E, logits=logits)
    ws = torch.full((moe.moe_ffn_few_workspace_bytes(T, H, I, E, k),), 0xFF, dtype=torch.uint8, device="cuda")
    ids = L.routing()[0].cpu()
    most = 1 if T == 1 else (8 if T * k > 2 * E else 4)
    held = {e: torch.nonzero(ids.view(-1) == e).view(-1).tolist() for e in (ids[0] if T == 1 else torch.unique(ids)).tolist()}
    if E >= 80:
        over = [i for i, rows in enumerate(held.values()) if len(rows) > most]
        assert over[0] < 64 <= over[-1]
    want = [(e, rows[:most]) for e, rows in held.items()]
    want += [(e, rows[at:at + most]) for e, rows in held.items() for at in range(most, len(rows), most)]
    y = L.run(workspace=ws)
    assert _table(ws, T, k, I) == want
    L.check(y)
    for _ in range(8):
        assert torch.equal(L.run(workspace=ws), y) and _table(ws, T, k, I) == want
