"""The group-normalisation reference itself, on the CPU: torch's own float64
group_norm and activations, and its gradients against automatic
differentiation and central differences."""
import pytest
import torch

import dropout_ref
import group_ref as ref


def _case(B=2, S=5, C=24, G=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(B, S, C) + r(C), 1 + 0.3 * r(C), 0.3 * r(C), r(B, S, C)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_forward_is_torch_group_norm(name):
    x, g, b, _ = _case()
    y, rstd, mean, _ = ref.forward(x, g, b, 3, 1e-5, name)
    t = torch.nn.functional.group_norm(x.transpose(1, 2), 3, g, b, 1e-5).transpose(1, 2)
    t = {"none": lambda v: v, "silu": torch.nn.functional.silu,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name](t)
    assert torch.allclose(y, t, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward_is_the_gradient(name, p):
    x, g, b, dy = _case(seed=1)
    fac = None
    if p:
        fac = dropout_ref.keep(x.shape, p, 5, 6).double() * 65536 / (65536 - dropout_ref.threshold(p))
    mean, rstd = ref.stats(x, 3, 1e-5)
    got = ref.backward(dy, x, g, b, rstd, mean, 3, name, fac)[:3]
    leaves = [t.clone().requires_grad_() for t in (x, g, b)]
    y = ref.forward(*leaves, 3, 1e-5, name, fac)[0]
    want = torch.autograd.grad((y * dy).sum(), leaves)
    for u, v in zip(got, want):
        assert torch.allclose(u, v, rtol=1e-9, atol=1e-10)
    # central differences of sum(y dy) at a few places
    h = 1e-6
    loss = lambda a, c, d: (ref.forward(a, c, d, 3, 1e-5, name, fac)[0] * dy).sum()  # noqa: E731
    for i in ((0, 0, 0), (1, 4, 23), (0, 2, 9)):
        e = torch.zeros_like(x)
        e[i] = h
        diff = (loss(x + e, g, b) - loss(x - e, g, b)) / (2 * h)
        assert abs(diff - got[0][i]) < 1e-6 * (1 + abs(diff))
    for c in (0, 11, 23):
        e = torch.zeros_like(g)
        e[c] = h
        assert abs((loss(x, g + e, b) - loss(x, g - e, b)) / (2 * h) - got[1][c]) < 1e-5
        assert abs((loss(x, g, b + e) - loss(x, g, b - e)) / (2 * h) - got[2][c]) < 1e-5
