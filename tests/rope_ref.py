"""Normalisation and rotation of query and key heads in float64 torch, from the
definitions, with the magnitudes that the CUDA path's tolerances multiply.

Tolerances.  An output of type t is rounded once, at most u_t = finfo(t).eps / 2
of its value.  In front of that stands float32 arithmetic on magnitudes bounded
by the terms that enter (`*_mag` below): a row's sums take at most 24 values in
a lane (three units of two chunks of four), two side by side, so 12 additions one
behind the other and one more, then 5 levels of shuffles and the product with 1 / D,
each rounding 2^-24 of the sum of magnitudes: 19 x 2^-24 for the mean, and one more
for the squares (half of it in rstd, and 2 ulp of the root): 12 x 2^-24.  The angle
is a 32-bit fraction of a turn, off by 2^-32 turns (and by 2^-25 radians at far
positions, tests/test_rope_far.py), rounded to 24 bits as turns and as radians, below
an eighth of a turn: 2 x 2^-24 radians; the polynomials add 2^-28 and two roundings:
cos and sin are off by at most 5 x 2^-24.  Six products and sums per element follow.  Together below
64 x 2^-24 = 2^-18 for y.  dx chains two such sums more and the products of two such
factors: 2^-16.  dgamma and dbeta add up to 64 rows in a thread (the tests' shapes)
and the rows of the CTAs, 32 side by side: 2^-16.
"""
import torch

ARITH_Y = 2.0 ** -18
ARITH_G = 2.0 ** -16


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def sections(pairs, axes):
    if axes == 1:
        return None
    if axes == 2:
        return (pairs - pairs // 2, pairs // 2)
    s = pairs // axes
    return (pairs - (axes - 1) * s,) + (s,) * (axes - 1)


def angles(pos, inv_freq, sec):
    """[T, pairs] in float64."""
    if sec is None:
        return pos.reshape(-1)[:, None].double() * inv_freq
    rows = pos.reshape(len(sec), -1).double()
    which = torch.tensor([a for a, n in enumerate(sec) for _ in range(n)], device=pos.device)
    return rows[which].t() * inv_freq


def pair_index(rd, inter, device):
    p = torch.arange(rd // 2, device=device)
    return (2 * p, 2 * p + 1) if inter else (p, p + rd // 2)


def rotate(v, ang, inter, mag=False):
    """Rows v [T, H, D] turned by ang [T, pairs]; mag: sums of magnitudes."""
    i, j = pair_index(2 * ang.shape[1], inter, v.device)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    out = v.clone()
    if mag:
        out[..., i] = v[..., i] + v[..., j]
        out[..., j] = out[..., i]
    else:
        out[..., i] = v[..., i] * c - v[..., j] * s
        out[..., j] = v[..., j] * c + v[..., i] * s
    return out


def norm(x, gamma, beta, eps, layer):
    """n, and the magnitudes of its terms."""
    x = x.double()
    if gamma is None:
        return x, x.abs()
    mean = x.mean(-1, keepdim=True) if layer else torch.zeros_like(x[..., :1])
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps) ** -0.5
    mag = x.abs() + x.abs().mean(-1, keepdim=True) if layer else x.abs()
    n, m = (x - mean) * rstd * gamma.double(), mag * rstd * gamma.double().abs()
    if beta is not None:
        n, m = n + beta.double(), m + beta.double().abs()
    return n, m


def forward(x, ang, inter, gamma=None, beta=None, eps=1e-6, layer=False):
    """y and its magnitudes, for x [T, H, D]."""
    n, m = norm(x, gamma, beta, eps, layer)
    return rotate(n, ang, inter), rotate(m, ang, inter, mag=True)


def backward(dy, x, ang, inter, gamma=None, eps=1e-6, layer=False):
    """(dx, dgamma, dbeta) and their magnitudes."""
    dn, dm = rotate(dy.double(), -ang, inter), rotate(dy.double().abs(), ang, inter, mag=True)
    if gamma is None:
        return (dn, None, None), (dm, None, None)
    x = x.double()
    mean = x.mean(-1, keepdim=True) if layer else torch.zeros_like(x[..., :1])
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps) ** -0.5
    xhat = (x - mean) * rstd
    xm = (x.abs() + x.abs().mean(-1, keepdim=True) if layer else x.abs()) * rstd
    g, gm = dn * gamma.double(), dm * gamma.double().abs()
    dx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    mag = gm + xm * (gm * xm).mean(-1, keepdim=True)
    if layer:
        dx, mag = dx - g.mean(-1, keepdim=True), mag + gm.mean(-1, keepdim=True)
    return ((rstd * dx, (dn * xhat).sum((0, 1)), dn.sum((0, 1))),
            (rstd * mag, (dm * xm).sum((0, 1)), dm.sum((0, 1))))


def check(got, want, mag, arith, what):
    """One rounding of got's type, and `arith` of the magnitudes."""
    tol = unit(got.dtype) * want.abs() + arith * mag
    if got.dtype == torch.float16:  # below the normal range the step is constant
        tol = tol + 2.0 ** -25
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        at = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what} at {at}: got {got[tuple(at)].item()}, want "
                             f"{want[tuple(at)].item()}, off by {err[tuple(at)].item():.3g}, "
                             f"allowed {tol[tuple(at)].item():.3g} ({int(bad.sum())} values)")
