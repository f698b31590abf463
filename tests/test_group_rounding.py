"""How far fp32 group normalisation is rounded, at data whose sums are exact.

Every channel of a group is constant over the positions, +a for its even
channels and -a for the odd ones, a = (1, 3 or 5) 2^k and an even number of
channels per group.  Block means, merges and folds then meet equal or opposite
values only, and the squared deviations are integer multiples of a^2 below
2^24 of them, so mean = 0 and M2 = S D a^2 carry no rounding whatever the
order of the sums.  With u = 2^-24 (half a step, relative) what is left is

  rstd   the quotient M2 / (S D) is exactly a^2; adding eps rounds once (u of
         the sum, so u / 2 of its root), the reciprocal root once: 1.5 u
  y      rstd gamma rounds once more, the multiply-add once: 2.5 u |xhat
         gamma| + u |y|
  SiLU   |act'| <= 1.1 times the error of z, and of the sigmoid s of k = z: the
         exponential's argument k log2(e) is off by 2 u relative (constant and
         product) and its result by 2 steps (4 u), which reach s times 1 - s;
         then 1 + e, the product of two denominators, the reciprocal (one
         step, 2 u) and the product with the other denominator, 5 u; z s is
         one more: |y| (6 u + (1 - s) (2 |k| + 4) u)

each times 1 + 2^-10 for products of these.
"""
import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SLACK = 1 + 2.0 ** -10
# a single position, odd counts of positions, one CTA per sample, clusters,
# several slabs; the last two large enough for the whole-GPU form
SHAPES = [(2, 1, 64, 8), (3, 7, 48, 4), (3, 49, 80, 8), (2, 100, 320, 32), (3, 1517, 168, 12),
          (1, 64, 1280, 32), (9, 333, 96, 12), (1, 60000, 64, 8), (2, 9000, 640, 64)]
EPS = [1e-5, 3e-3, 0.7]


def _case(B, S, C, G):
    D = C // G
    assert D % 2 == 0 and S * D * 25 < 1 << 24
    i = torch.arange(B * G)
    a = ((1 + 2 * (i % 3)) * torch.exp2((i % 7 - 4).float())).view(B, 1, G, 1)
    sign = (1 - 2 * (torch.arange(D) % 2)).view(1, 1, 1, D)
    x = (a * sign).expand(B, S, G, D).reshape(B, S, C).float()
    g = torch.Generator().manual_seed(C + S)
    gamma, beta = 1 + 0.3 * torch.randn(C, generator=g), torch.randn(C, generator=g)
    return x.cuda(), gamma.cuda(), beta.cuda(), a.view(B, G).double().cuda()


@pytest.mark.parametrize("form", [None, 0, 1, 2])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_of_exact_statistics(shape, form, monkeypatch):
    B, S, C, G = shape
    x, gamma, beta, a = _case(*shape)
    if form is not None:
        monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
        try:
            gb.norm_group_plan(B, S, C, G, gb.FP32)
        except gb.NormError:
            pytest.skip("too large for this form")
    for eps in EPS:
        eps64 = torch.tensor(eps, dtype=torch.float32).double().item()
        y, rstd, mean = gb.norm_group_fwd(x, gamma, beta, G, eps)
        want = 1 / torch.sqrt(a * a + eps64)
        assert torch.equal(mean, torch.zeros_like(mean))
        err = ((rstd.double() - want) / want).abs().max().item()
        assert err <= 1.5 * U * SLACK, f"rstd off by {err / U:.2f} half steps at eps {eps}"
        spread = want[:, None, :, None].expand(B, S, G, C // G).reshape(B, S, C)
        xg = x.double() * spread * gamma.double()
        z = xg + beta.double()
        ez = 2.5 * U * xg.abs() + U * z.abs()
        over = ((y.double() - z).abs() - ez * SLACK).max().item()
        assert over <= 0, f"y beyond its bound by {over}"
        y, _, _ = gb.norm_group_fwd(x, gamma, beta, G, eps, "silu")
        s = torch.sigmoid(z)
        bound = 1.1 * ez + (z * s).abs() * U * (6 + (1 - s) * (2 * z.abs() + 4))
        over = ((y.double() - z * s).abs() - bound * SLACK).max().item()
        assert over <= 0, f"SiLU y beyond its bound by {over}"


@pytest.mark.parametrize("form", [None, 0, 1, 2])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient_of_a_constant_vanishes(shape, form, monkeypatch):
    """gamma = 1, rstd a power of two, mean = 0 and dy one integer per group:
    the sums of dy are exact, those of dy xhat are 0, and the mean of dy is dy
    itself, so dx = rstd (dy - dy) = 0 without a rounding."""
    B, S, C, G = shape
    x, _, _, a = _case(*shape)
    D = C // G
    ones = torch.ones(C, device="cuda")
    i = torch.arange(B * G, device="cuda")
    rstd = torch.exp2((i % 5 - 2).float()).view(B, G)
    dy = (1 + i % 3).float().view(B, 1, G, 1).expand(B, S, G, D).reshape(B, S, C).contiguous()
    if form is not None:
        monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
        try:
            gb.norm_group_plan(B, S, C, G, gb.FP32, True)
        except gb.NormError:
            pytest.skip("too large for this form")
    dx, dg, db = gb.norm_group_bwd(dy, x, ones, None, rstd, torch.zeros_like(rstd), G)
    assert torch.equal(dx, torch.zeros_like(dx)), dx.abs().max().item()
    assert torch.equal(db, dy.sum((0, 1)))


@pytest.mark.parametrize("c", [3.0, -7.0, 41.0])
@pytest.mark.parametrize("S", [3, 41, 47, 61, 83, 1001])
def test_mean_of_a_constant_is_that_constant(S, c):
    """Sums of an integer times the count are exact, and so is the quotient."""
    x = torch.full((2, S, 48), c, device="cuda")
    one = torch.ones(48, device="cuda")
    for G in (1, 4, 16):
        y, rstd, mean = gb.norm_group_fwd(x, one, None, G, 1e-4)
        assert torch.equal(mean, torch.full_like(mean, c)), (S, G)
        assert torch.equal(y, torch.zeros_like(y))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("big", [1e3, 1e8, 1e15])
def test_large_activations_dx(act, big):
    """dx where the sigmoid saturates and z k'(z) overflows: finite, and within
    the general tolerance of the 64-bit gradient."""
    import group_ref as ref

    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, g, b, dy = r(1, 16, 16), (1 + 0.2 * r(16)) * big, r(16), r(1, 16, 16)
    y, rstd, mean = gb.norm_group_fwd(x, g, b, 2, 1e-5, act)
    dx, _, _ = gb.norm_group_bwd(dy, x, g, b, rstd, mean, 2, act)
    assert torch.isfinite(dx).all()
    want = ref.backward(dy, x, g, b, rstd, mean, 2, act)
    ref.check(dx, want[0], want[3], f"{act} {big} dx")


@pytest.mark.parametrize("form", [0, 1, 2])
def test_infinities_in_statistics_and_sums(form, monkeypatch):
    """A variance that overflows gives rstd = 0 and y = beta; an infinite dy
    gives the infinities and NaN of dx = rstd (g - mean(g) - xhat mean(g xhat))
    in its group, and none outside."""
    monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
    B, S, C, G = 2, 60, 64, 4
    gen = torch.Generator().manual_seed(form)
    x, dy = (torch.randn(B, S, C, generator=gen).cuda() for _ in range(2))
    gamma, beta = (torch.randn(C, generator=gen).cuda() for _ in range(2))
    huge = x.clone()
    huge[1, :, :16] = 1e20 * torch.sign(x[1, :, :16])
    y, rstd, mean = gb.norm_group_fwd(huge, gamma, beta, G)
    assert (rstd[1, 0] == 0) and torch.equal(y[1, :, :16], beta[:16].expand(S, 16))
    assert torch.isfinite(y).all() and (rstd.view(-1)[:4] > 0).all()
    y, rstd, mean = gb.norm_group_fwd(x, gamma, beta, G)
    clean = gb.norm_group_bwd(dy, x, gamma, beta, rstd, mean, G)[0]
    for value in (float("inf"), -float("inf")):
        d = dy.clone()
        d[0, 11, 21] = value  # group 1
        dx, dg, db = gb.norm_group_bwd(d, x, gamma, beta, rstd, mean, G)
        xhat = ((x[0, :, 16:32] - mean[0, 1]) * rstd[0, 1]).double()
        g = d[0, :, 16:32].double() * gamma[16:32].double()
        want = rstd[0, 1].double() * (g - g.mean() - xhat * (g * xhat).mean())
        got = dx[0, :, 16:32].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
        dx[0, :, 16:32] = clean[0, :, 16:32] = 0
        assert torch.equal(dx, clean)
        assert db[21].item() == value and not torch.isfinite(dg[21])
