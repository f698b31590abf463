"""Group normalisation + activation (+ dropout) in float64 torch, from the
definitions, with the tolerances of the CUDA path.

Tolerances (relative to magnitudes that bound each quantity's terms): an
output of type t is rounded once, at most u_t = finfo(t).eps / 2 of its value
(u = 0 for the fp32 outputs' final rounding, which the arithmetic term
covers); the float32 arithmetic in front of it is held to 2^-16 of the sum of
the magnitudes of the terms that enter.  Where that comes from: the running
mean of a thread takes one merge per four rows, each with a rounding of 2^-24
of the mean's magnitude; the shapes tested have at most 70 merges in a row
plus at most 20 levels of folds, 90 x 2^-24 < 2^-17; the squared deviations
and rstd add as much again relative to themselves, and the affine, the
exponential (2 + |1.17 k| ulp), the quotient and the products below 2^-19.
"""
import math

import torch

ARITH = 2.0 ** -16


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def act(z, name):
    if name == "none":
        return z
    if name == "silu":
        return z / (1 + torch.exp(-z))
    c = math.sqrt(2 / math.pi)
    return 0.5 * z * (1 + torch.tanh(c * (z + 0.044715 * z ** 3)))


def act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def stats(x, G, eps):
    B, C = x.shape[0], x.shape[-1]
    xg = x.double().reshape(B, -1, G, C // G)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    return mean, 1 / torch.sqrt(var + eps)


def spread(v, x, G):
    """[B, G] -> the shape [B, S, C] of x."""
    B, S, C = x.shape
    return v[:, None, :, None].expand(B, S, G, C // G).reshape(B, S, C)


def forward(x, gamma, beta, G, eps, name, fac=None):
    """y, rstd, mean and the magnitude that ARITH multiplies for y."""
    mean, rstd = stats(x, G, eps)
    mu, rs = spread(mean, x, G), spread(rstd, x, G)
    xhat = (x.double() - mu) * rs
    g, b = gamma.double(), 0.0 if beta is None else beta.double()
    z = xhat * g + b
    y = act(z, name)
    babs = 0.0 if beta is None else b.abs()
    mag = g.abs() * (xhat.abs() + mu.abs() * rs + 1) + babs
    if fac is not None:
        y, mag = y * fac, mag * fac
    return y, rstd, mean, mag


def backward(dy, x, gamma, beta, rstd, mean, G, name, fac=None):
    """dx, dgamma, dbeta at the given statistics, and their magnitudes."""
    B, S, C = x.shape
    mu, rs = spread(mean.double(), x, G), spread(rstd.double(), x, G)
    xhat = (x.double() - mu) * rs
    g, b = gamma.double(), 0.0 if beta is None else beta.double()
    z = xhat * g + b
    d = dy.double() if fac is None else dy.double() * fac
    dz = d * act_grad(z, name)
    gm = lambda v: spread(v.reshape(B, S, G, C // G).mean((1, 3)), x, G)  # noqa: E731
    gz = dz * g
    dx = rs * (gz - gm(gz) - xhat * gm(gz * xhat))
    # magnitudes: |dy| times what can multiply an error of z
    xm = xhat.abs() + mu.abs() * rs * 2.0 ** -4
    da = d.abs() * (1 + g.abs() * xm + (0.0 if beta is None else b.abs()))
    ga = da * g.abs()
    mx = rs * (ga + gm(ga) + xm * gm(ga * xm))
    return (dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1)),
            mx, (da * xm).sum((0, 1)), da.sum((0, 1)))


def check(got, ref, mag, name):
    u = unit(got.dtype)
    err = (got.double() - ref).abs()
    bound = u * ref.abs() + ARITH * mag
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a subnormal step
    bad = ~(err <= bound)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of tolerance, first at "
                             f"{i}: got {got[tuple(i)].item()!r} want {ref[tuple(i)].item()!r} "
                             f"bound {bound[tuple(i)].item():.3g}")
