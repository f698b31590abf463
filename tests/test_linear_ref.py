"""The float64 form of the linear layer: against torch's own functions, autograd
and differences (CPU)."""
import pytest
import torch

import linear_ref as lr


def _case(seed=0, M=5, K=7, N=6):
    g = torch.Generator().manual_seed(seed)
    r = dict(generator=g, dtype=torch.float64)
    return (torch.randn(M, K, **r), torch.randn(N, K, **r), torch.randn(N, **r),
            torch.randn(M, N, **r), torch.randn(M, N, **r))


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_forward_and_gradients(name):
    x, w, b, r, dy = _case()
    fn = {"none": lambda t: t, "silu": torch.nn.functional.silu,
          "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[name]
    (y, z), _ = lr.forward(x, w, b, r, name)
    assert torch.allclose(z, torch.nn.functional.linear(x, w, b), atol=1e-13)
    assert torch.allclose(y, r + fn(z), atol=1e-13)
    ins = [t.clone().requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad(fn(torch.nn.functional.linear(*ins)), ins, dy)
    got, _, _ = lr.backward(dy, x, w, z, name)
    for a, c in zip(got, want):
        assert torch.allclose(a, c, atol=1e-12)
    for k in range(3):
        d = torch.randn(ins[k].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(k))
        h = 1e-6
        args = [[x, w, b], [x, w, b]]
        args[0][k], args[1][k] = (x, w, b)[k] + h * d, (x, w, b)[k] - h * d
        up, dn = (lr.forward(*a, r, name)[0][0] for a in args)
        slope = ((up - dn) * dy).sum() / (2 * h)
        assert abs(slope - (got[k] * d).sum()) < 1e-6 * (1 + abs(slope))


def test_slope_bound():
    z = torch.linspace(-12, 12, 100001, dtype=torch.float64)
    for name in ("silu", "gelu"):
        assert lr.act_grad(z, name)[0].abs().max() < lr.act_slope


def test_check_sees_wrong_results():
    x, w, b, r, _ = (t.bfloat16() for t in _case(1, 70, 40, 66))
    (y, z), (ey, ez) = lr.forward(x, w, b, r, "gelu")
    lr.check(y.bfloat16(), y, ey, "y")
    lr.check(z.bfloat16(), z, ez, "z")
    for wrong in (y - r.double(), y * 1.01, y.roll(1, 0), lr.forward(x, w, None, r, "gelu")[0][0],
                  lr.forward(x, w, b, r, "silu")[0][0], y.bfloat16().double() * (1 + 2.0 ** -7)):
        with pytest.raises(AssertionError):
            lr.check(wrong.bfloat16(), y, ey, "y")
