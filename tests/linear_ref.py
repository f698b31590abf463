"""The linear layer with bias, activation and residual in float64 torch, from
the definitions, with the tolerances of the CUDA path.

Tolerances.  An output of type t is rounded once, at most u_t = finfo(t).eps / 2
of its value.  Products of two 16-bit values are exact in fp32; a sum of K of
them in fp32, in any order, with or without rounding to nearest, is off by at
most K 2^-23 of the sum of their magnitudes S.  Activations have slopes below
1.13; their exponential, sum and quotient take up to 2^-20 of the result
(exponents up to 88 scaled by log2 e: 88 x 1.44 x 2^-24 absolute in the
exponent, below 2^-17 relative where the result is below 1e-30 of z, and 2^-20
where the exponent is below 16).  dz is rounded once more for the products (u_t
of each term), its activation slope is off by at most 2^-18 of the magnitudes of
its two terms.  These bounds hold for every element; the RMS error, which would
show a missing or doubled term that they leave room for, is held to 1.25 times
the size that independent roundings give, u / sqrt(3) of the rounded values
(a relative rounding error is uniform in at most +-u), plus the fp32 part.
"""
import math

import torch

act_slope = 1.13


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def act(z, name):
    if name == "none":
        return z
    if name == "silu":
        return z * torch.sigmoid(z)
    # (1 + tanh(u)) / 2 = sigmoid(2 u), which keeps its digits where tanh(u) is -1
    # in float64 (z < -8.3, where the result is still 1e-24 and less of z)
    c = 2 * math.sqrt(2 / math.pi)
    return z * torch.sigmoid(c * (z + 0.044715 * z ** 3))


def act_grad(z, name):
    """act'(z) and the magnitudes of its two terms."""
    if name == "none":
        return torch.ones_like(z), torch.ones_like(z)
    if name == "silu":
        s = torch.sigmoid(z)
        b = z * s * (1 - s)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        b = z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    return s + b, s + b.abs()


def forward(x, w, bias, r, name):
    """(y, z) and the fp32 error bounds in front of their rounding."""
    x, w = x.double(), w.double()
    K = x.shape[-1]
    z = x @ w.t()
    ez = K * 2.0 ** -23 * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -23 * z.abs()
    y = act(z, name)
    ey = act_slope * ez + (2.0 ** -20 * y.abs() if name != "none" else 0)
    if r is not None:
        y = y + r.double()
        ey = ey + 2.0 ** -23 * (y.abs() + r.double().abs())
    return (y, z), (ey, ez)


def backward(dy, x, w, z, name):
    """(dx, dw, dbias), bounds on their errors in front of the last rounding, and
    the squares of those that the rounding of dz gives on average."""
    dyd, x, w = dy.double(), x.double(), w.double()
    M, N = dyd.shape
    slope, mag = act_grad(z.double(), name) if name != "none" else (1.0, 0.0)
    dz = dyd * slope
    u = unit(dy.dtype) if name != "none" else 0.0
    edz = u * dz.abs() + (2.0 ** -18 * dyd.abs() * mag if name != "none" else 0)
    edx = edz @ w.abs() + N * 2.0 ** -23 * (dz.abs() @ w.abs())
    edw = edz.t() @ x.abs() + M * 2.0 ** -23 * (dz.abs().t() @ x.abs())
    edb = 2.0 ** -16 * (dyd.abs() * (mag if name != "none" else 1.0)).sum(0)
    sq = u * u / 3
    return ((dz @ w, dz.t() @ x, dz.sum(0)), (edx, edw, edb),
            (sq * (dz.square() @ w.square()), sq * (dz.square().t() @ x.square())))


def check(got, want, err, what, square=None):
    """Every element within its rounding and `err`; the RMS error within 1.25 times
    the expected one.  square: what other roundings add to its square."""
    u = unit(got.dtype) if got.dtype != torch.float32 else 2.0 ** -24
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0  # subnormal steps
    off = (got.double() - want).abs()
    tol = u * want.abs() * (1 + 2.0 ** -10) + err * (1 + u) + tiny
    bad = ~(off <= tol)
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what} at {at}: got {got[at].item()}, want {want[at].item()}, off by "
                             f"{off[at].item():.3g}, allowed {tol[at].item():.3g} "
                             f"({int(bad.sum())} of {bad.numel()} values)")
    if want.numel() >= 4096 and got.dtype != torch.float32:
        sq = u * u / 3 * want.square() + (square if square is not None else 0)
        fp32 = (err if square is None else 2.0 ** -16 * want.abs()).square().mean().sqrt().item()
        most = 1.25 * sq.mean().sqrt().item() + fp32 + tiny
        rms = off.square().mean().sqrt().item()
        assert rms <= most, f"{what}: RMS error {rms:.3g}, expected below {most:.3g}"
