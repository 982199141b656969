"""References of the ragged products in 64 bits, and their error bounds.

A sum of K products in fp32 by any order of additions of depth d is off by at most d * 2^-23 * sum |a w|
(2^-24 a rounded addition, doubled for matrix instructions that cut instead of rounding).  A matrix
instruction takes 32 products a step, so d <= K / 32 + 32.  Storing rounds by half a step more."""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}


def sum_bound(K, mass):
    return (K / 32 + 32) * 2.0 ** -23 * mass


def assert_close(got, ref, err, label=""):
    """|got - ref| <= err (before storing) + half a step of the output's type."""
    dt = got.dtype
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    tol = err + HALF_STEP[dt] * (ref.abs() + err) + TINY[dt]
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (label, int(bad.sum()), float((off / tol).nan_to_num(float("inf")).max()))


def offsets_of(counts, device="cuda"):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
    return o.to(device)


def silu_mul(G):
    g, u = G.chunk(2, dim=-1)
    return g * torch.sigmoid(g) * u


def silu_bound(G, err):
    """Error of silu(g) * u from errors err of g and u: |silu'| <= 1.1, and the fast exponential and quotient
    are off by less than 2^-18 relative for |g| <= 30 (the argument's rounding, |g| * 1.5 * 2^-24, leads)."""
    g, u = G.chunk(2, dim=-1)
    eg, eu = err.chunk(2, dim=-1)
    s = (g * torch.sigmoid(g)).abs()
    return 1.1 * eg * (u.abs() + eu) + s * eu + 2.0 ** -18 * s * u.abs()


def grouped(A, W, counts):
    """(C, mass): rows of A in group order times their expert's W^T, in 64 bits, and the sums of magnitudes."""
    C = torch.zeros((A.shape[0], W.shape[1]), dtype=torch.float64, device=A.device)
    mass = torch.zeros_like(C)
    at = 0
    for e, n in enumerate(counts):
        if n:
            a, w = A[at:at + n].double(), W[e].double()
            C[at:at + n] = a @ w.t()
            mass[at:at + n] = a.abs() @ w.abs().t()
        at += n
    return C, mass


def grouped_dw(dC, A, counts):
    E = len(counts)
    dW = torch.zeros((E, dC.shape[1], A.shape[1]), dtype=torch.float64, device=A.device)
    mass = torch.zeros_like(dW)
    at = 0
    for e, n in enumerate(counts):
        if n:
            d, a = dC[at:at + n].double(), A[at:at + n].double()
            dW[e] = d.t() @ a
            mass[e] = d.abs().t() @ a.abs()
        at += n
    return dW, mass
