"""The linear layer's long contractions, also where the output is small: a missing or
doubled part of the sum must show.

The RMS error of an output of a few hundred elements or more is held to 1.25 times
what independent roundings give, u / sqrt(3) of the rounded values, plus that of the
fp32 sums, for which the terms' signs count: with R = sqrt(sum of the squares of the
K terms), a partial sum is 2/3 R in the mean over the way of a random walk.  A tensor
instruction adds 16 products to it; taking its adder to lose up to four units of the
last place (2^-23) of the partial sum, always in the same direction, K / 16
instructions, up to 8 joins and the bias are off by (K / 16 + 9) 2^-21 2/3 R.  (A
relative rounding error uniform in +-u is the worst of a binade; over random values
it is 0.73 of that, and the mean square of 128 products of normal values with uniform
errors is spread by 19 %, its root by 9 %: 1.25 is 7 such spreads away.)
A block of 64 terms left out is off by sqrt(64 / K) R: 0.022 R for the longest
contraction here, where the roundings of bf16 allow 0.0066 R with two of them."""
import math

import pytest
import torch

import linear_ref as lr
import memory_bound_normalization_rmsnorm_gb300 as gb
from test_linear import DT, SHAPES, _make

LEAST = 128  # elements that an RMS error is taken over


def sum_rms(K, squares):
    """RMS error of fp32 sums of K terms; squares: of the terms, summed."""
    return (K / 16 + 9) * 2.0 ** -21 * 2 / 3 * squares.mean().sqrt().item()


def most_rms(want, dtype, fp32, square=None):
    u = lr.unit(dtype)
    sq = u * u / 3 * want.square()
    if square is not None:
        sq = sq + square
    return 1.25 * sq.mean().sqrt().item() + fp32 + (2.0 ** -25 if dtype == torch.float16 else 0)


def check_rms(got, want, most, what):
    if want.numel() < LEAST:
        return
    rms = (got.double() - want).square().mean().sqrt().item()
    assert rms <= most, f"{what}: RMS error {rms:.3g}, expected below {most:.3g}"


def forward_limits(x, w, bias, r, name):
    """(y, z), and the RMS errors that they may have."""
    (y, z), _ = lr.forward(x, w, bias, r, name)
    fp32 = sum_rms(x.shape[1], x.double().square() @ w.double().square().t())
    arith = 2.0 ** -20 * (y.square().mean().sqrt().item() + r.double().square().mean().sqrt().item())
    return (y, z), (most_rms(y, x.dtype, lr.act_slope * fp32 + arith), most_rms(z, x.dtype, fp32))


def backward_limits(dy, x, w, z, name):
    """(dx, dw, dbias), and the RMS errors that they may have.  The slope of an
    activation is off by up to 2^-18 of its terms' magnitudes, in dz one by one."""
    want, _, sq = lr.backward(dy, x, w, z, name)
    mag = lr.act_grad(z.double(), name)[1] if name != "none" else torch.ones_like(z, dtype=torch.float64)
    dz2, x2, w2 = (dy.double() * mag).square(), x.double().square(), w.double().square()
    M, N = dy.shape
    most = [most_rms(want[0], dy.dtype, sum_rms(N, dz2 @ w2) + 2.0 ** -18 * (dz2 @ w2).mean().sqrt().item(), sq[0]),
            most_rms(want[1], dy.dtype, sum_rms(M, dz2.t() @ x2) + 2.0 ** -18 * (dz2.t() @ x2).mean().sqrt().item(),
                     sq[1]),
            # fp32 additions one after the other, rounded to nearest: a random walk
            (2.0 ** -24 * (math.sqrt(M) + 1) + 2.0 ** -18) * dz2.sum(0).mean().sqrt().item()]
    return want, most


def _host(dtype, M, K, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DT[dtype]
    return dict(x=r(M, K).to(dt), w=(r(N, K) / K ** 0.5).to(dt), bias=(0.3 * r(N)).to(dt),
                r=r(M, N).to(dt), dy=r(M, N).to(dt))


def _parts(K):
    """Terms that a fault could leave out: a block of 64 (the first, the last), an
    eighth."""
    nk = (K + 63) // 64
    cuts = {(0, min(64, K)), ((nk - 1) * 64, K), (K // 8 // 64 * 64, max(K // 4 // 64 * 64, 64))}
    return [(a, min(b, K)) for a, b in cuts if a < K and b > a]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,name", [("bf16", "none"), ("bf16", "gelu"), ("fp16", "silu")])
def test_missing_terms_show(shape, dtype, name):
    """The limits take the right result, rounded, and refuse it without some terms
    (CPU).  The last block of a K that is no multiple of 64 has as few as one term:
    looked at where it weighs as much as 64 of the longest contraction here."""
    M, K, N = shape
    c = _host(dtype, *shape)
    dt, seen = c["x"].dtype, 0
    (y, z), (ly, lz) = forward_limits(c["x"], c["w"], c["bias"], c["r"], name)
    check_rms(y.to(dt), y, ly, "y")
    check_rms(z.to(dt), z, lz, "z")
    zr = z.to(dt)
    (dx, dw, db), (ldx, ldw, ldb) = backward_limits(c["dy"], c["x"], c["w"], zr, name)
    dz = c["dy"].double() * (lr.act_grad(zr.double(), name)[0] if name != "none" else 1.0)
    for t, most in ((dx, ldx), (dw, ldw)):
        check_rms(t.to(dt), t, most, "gradient")
    check_rms(db.float(), db, ldb, "dbias")
    x, w = c["x"].double(), c["w"].double()

    def refused(got, want, most, weight):
        nonlocal seen
        if want.numel() < LEAST or weight < 64 / 131072:
            return
        seen += 1
        with pytest.raises(AssertionError):
            check_rms(got, want, most, "mutant")

    for a, b in _parts(K):
        cut = z - x[:, a:b] @ w[:, a:b].t()
        refused(cut.to(dt), z, lz, (b - a) / K)
        refused((lr.act(cut, name) + c["r"].double()).to(dt), y, ly, (b - a) / K)
    for a, b in _parts(N):
        refused((dx - dz[:, a:b] @ w[a:b]).to(dt), dx, ldx, (b - a) / N)
    for a, b in _parts(M):
        refused((dw - dz[a:b].t() @ x[a:b]).to(dt), dw, ldw, (b - a) / M)
        refused((db - dz[a:b].sum(0)).float(), db, ldb, (b - a) / M)
    assert seen > 0 or M * N < LEAST and M * K < LEAST


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_sums_are_whole(dtype, name, shape):
    c = _make(dtype, *shape)
    y, z = gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], name, want_z=True)
    want, most = forward_limits(c["x"], c["w"], c["bias"], c["r"], name)
    for n, g, t, m in zip("yz", (y, z), want, most):
        check_rms(g, t, m, n)
    zr = want[1].to(z.dtype)
    got = gb.norm_linear_bwd(c["dy"], c["x"], c["w"], zr if name != "none" else None, name)
    want, most = backward_limits(c["dy"], c["x"], c["w"], zr, name)
    for n, g, t, m in zip(("dx", "dw", "dbias"), got, want, most):
        check_rms(g, t, m, n)
    assert gb.norm_get_device_error() == 0
