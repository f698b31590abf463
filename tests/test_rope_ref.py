"""The float64 form of the head normalisation and rotation: against closed
forms, autograd and differences (CPU)."""
import math

import pytest
import torch

import rope_ref as rr


def _case(axes, seed=0, T=5, H=3, D=24, rd=16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g, dtype=torch.float64)
    gamma = 1 + 0.2 * torch.randn(D, generator=g, dtype=torch.float64)
    beta = 0.2 * torch.randn(D, generator=g, dtype=torch.float64)
    sec = rr.sections(rd // 2, axes)
    pos = torch.randint(-50, 1000, (T,) if axes == 1 else (axes, T), generator=g)
    inv = torch.tensor([100.0 ** (-2 * i / rd) for i in range(rd // 2)], dtype=torch.float64)
    return x, gamma, beta, rr.angles(pos, inv, sec)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(inter):
    x, _, _, _ = _case(1)
    inv = torch.tensor([0.3, 1.7, 0.01, 2.0, 0.5, 0.25, 1.0, 3.0], dtype=torch.float64)
    q, k = x[:1, :1].expand(7, 1, 24), x[1:2, 1:2].expand(7, 1, 24)
    a = rr.angles(torch.arange(7), inv, None)
    rq = rr.rotate(q, a, inter)
    assert torch.allclose(rq[..., :16].square().sum(-1), q[..., :16].square().sum(-1))
    assert torch.equal(rq[..., 16:], q[..., 16:])
    rk = rr.rotate(k, rr.angles(torch.arange(7) + 3, inv, None), inter)
    dots = (rq * rk).sum(-1)
    assert torch.allclose(dots, dots[:1].expand_as(dots))  # depends on the distance alone


def test_pairs_and_quarter_turn():
    v = torch.arange(1.0, 7.0, dtype=torch.float64).view(1, 1, 6)
    a = torch.full((1, 2), math.pi / 2, dtype=torch.float64)
    assert torch.allclose(rr.rotate(v, a, False), torch.tensor([-3.0, -4, 1, 2, 5, 6]).double())
    assert torch.allclose(rr.rotate(v, a, True), torch.tensor([-2.0, 1, -4, 3, 5, 6]).double())


def test_sections_pick_the_axis():
    pos = torch.tensor([[1, 2], [10, 20], [100, 200]])
    a = rr.angles(pos, torch.ones(4, dtype=torch.float64), (2, 1, 1))
    assert a.tolist() == [[1, 1, 10, 100], [2, 2, 20, 200]]


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_backward_against_autograd_and_differences(kind, inter, axes):
    x, gamma, beta, ang = _case(axes)
    layer = kind == "layer"
    par = (None, None) if kind == "none" else (gamma, beta if layer else None)

    def f(x, gamma, beta):
        return rr.forward(x, ang, inter, gamma, beta, 1e-3, layer)[0]

    dy = torch.randn(x.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(9))
    got, _ = rr.backward(dy, x, ang, inter, par[0], 1e-3, layer)
    ins = [t.clone().requires_grad_() for t in (x, *par) if t is not None]
    full = ins + [None] * (3 - len(ins))
    want = torch.autograd.grad(f(*full), ins, dy)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, atol=1e-12)
    for k, t in enumerate(ins):
        d = torch.randn(t.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(k))
        h = 1e-6
        up, dn = list(full), list(full)
        up[k], dn[k] = (t + h * d).detach(), (t - h * d).detach()
        slope = ((f(*up) - f(*dn)) * dy).sum() / (2 * h)
        assert abs(slope - (got[k] * d).sum()) < 1e-6 * (1 + abs(slope))
