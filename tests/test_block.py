"""A pre-norm transformer block out of the library's calls, both directions: norm,
projection, head norm + rotation, attention (plain torch), projection back onto
the residual stream, norm, MLP.  Against the same block in float64 torch with
autograd."""
import math

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

T, C, H, HK, D, F = 150, 256, 4, 2, 64, 640
EPS = 1e-5


def _params(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, k=1.0: (k * torch.randn(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731
    return dict(g1=1 + r(C, k=0.1), wqkv=r((H + 2 * HK) * D, C, k=C ** -0.5), gq=1 + r(D, k=0.1),
                gk=1 + r(D, k=0.1), wo=r(C, H * D, k=(H * D) ** -0.5), bo=r(C, k=0.1),
                g2=1 + r(C, k=0.1), b2=r(C, k=0.1), wu=r(F, C, k=C ** -0.5), bu=r(F, k=0.1),
                wd=r(C, F, k=F ** -0.5), bd=r(C, k=0.1)), r(T, C), r(T, C)


def _attend(q, k, v):
    """Causal attention of [T, H, D] queries and [T, HK, D] keys and values."""
    k, v = (t.repeat_interleave(H // HK, 1) for t in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(D)
    s = s.masked_fill(torch.ones(T, T, device=q.device).triu(1).bool(), float("-inf"))
    return torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(T, H * D)


def _reference(p, h, pos, inv, sec):
    which = torch.tensor([a for a, n in enumerate(sec) for _ in range(n)], device=h.device)
    ang = pos.double()[which].t() * inv
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def rms(x, g):
        return x * (x.square().mean(-1, keepdim=True) + EPS) ** -0.5 * g

    def turn(x):
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    qkv = rms(h, p["g1"]) @ p["wqkv"].t()
    q, k, v = (t.reshape(T, -1, D) for t in qkv.split((H * D, HK * D, HK * D), 1))
    h = h + _attend(turn(rms(q, p["gq"])), turn(rms(k, p["gk"])), v) @ p["wo"].t() + p["bo"]
    y = torch.nn.functional.layer_norm(h, (C,), p["g2"], p["b2"], EPS)
    a = torch.nn.functional.gelu(y @ p["wu"].t() + p["bu"], approximate="tanh")
    return h + a @ p["wd"].t() + p["bd"]


def _run(p, h0, dout, pos, inv, sec):
    """Output and gradients by the library's calls."""
    y1, r1, _ = gb.norm_fwd(h0, p["g1"], None, EPS, gb.RMS)
    qkv, _ = gb.norm_linear_fwd(y1, p["wqkv"])
    q, k = qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + HK) * D].view(T, HK, D)
    rot = dict(eps=EPS, mode=gb.RMS, sections=sec)
    yq, yk = gb.norm_rope_fwd(q, k, pos, inv, p["gq"], p["gk"], **rot)
    # attention in plain torch, with its gradients by autograd
    leaves = [t.detach().float().requires_grad_() for t in
              (yq, yk, qkv[:, (H + HK) * D:].reshape(T, HK, D))]
    att = _attend(*leaves)
    o = att.detach().bfloat16()
    h1, _ = gb.norm_linear_fwd(o, p["wo"], p["bo"], h0)
    y2, r2, m2 = gb.norm_fwd(h1, p["g2"], p["b2"], EPS, gb.LAYER)
    a, z = gb.norm_linear_fwd(y2, p["wu"], p["bu"], None, "gelu", want_z=True)
    out, _ = gb.norm_linear_fwd(a, p["wd"], p["bd"], h1)

    gr = {}
    da, gr["wd"], gr["bd"] = gb.norm_linear_bwd(dout, a, p["wd"])
    dy2, gr["wu"], gr["bu"] = gb.norm_linear_bwd(da, y2, p["wu"], z, "gelu")
    dh1, gr["g2"], gr["b2"] = gb.norm_add_bwd(dy2, dout, h1, p["g2"], r2, m2, gb.LAYER)
    do, gr["wo"], gr["bo"] = gb.norm_linear_bwd(dh1, o, p["wo"])
    dyq, dyk, dv = (t.bfloat16() for t in torch.autograd.grad(att, leaves, do.float()))
    dqkv = torch.empty_like(qkv)
    _, _, gr["gq"], gr["gk"], _, _ = gb.norm_rope_bwd(
        dyq, dyk, q, k, pos, inv, p["gq"], p["gk"], **rot, dq=dqkv[:, :H * D].view(T, H, D),
        dk=dqkv[:, H * D:(H + HK) * D].view(T, HK, D))
    dqkv[:, (H + HK) * D:] = dv.reshape(T, -1)
    dy1, gr["wqkv"], _ = gb.norm_linear_bwd(dqkv, y1, p["wqkv"], want_dbias=False)
    gr["h"], gr["g1"], _ = gb.norm_add_bwd(dy1, dh1, h0, p["g1"], r1, None, gb.RMS)
    return out, gr


@pytest.mark.gpu
def test_block_both_directions():
    """Relative errors (2-norm).  Each bf16 rounding of a tensor is off by at most
    2^-8 / sqrt(3) of its values in the 2-norm, and a chain of n of them that pass
    through maps of gain up to g by sqrt(n) g times that; the longest chain here
    (out's gradient to wqkv and gq) has 14 roundings: sqrt(14) x 2^-8 / sqrt(3) =
    0.0084 with gain 1.  Normalisation and softmax backward passes subtract
    projections (gain up to 2): 0.017.  The residual stream alone carries a
    gradient of gain 1 past them."""
    p, h, dout = _params()
    pos = torch.stack([torch.arange(T), torch.arange(T) // 12, torch.arange(T) % 12]).cuda()
    sec = (8, 12, 12)
    inv = torch.tensor([10000.0 ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64).cuda()
    out, gr = _run(p, h, dout, pos, inv, sec)
    p64 = {n: t.double().requires_grad_() for n, t in p.items()}
    h64 = h.double().requires_grad_()
    want = _reference(p64, h64, pos, inv, sec)
    wgr = torch.autograd.grad(want, [*p64.values(), h64], dout.double())
    off = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    assert off(out, want) < 0.0084
    for n, w in zip([*p64, "h"], wgr):
        assert off(gr[n], w) < 0.017, n
    assert gb.norm_get_device_error() == 0


@pytest.mark.gpu
def test_block_replayed():
    """The same calls captured into a graph: the same bits, also for new inputs."""
    p, h, dout = _params()
    pos = torch.randint(0, 1 << 20, (3, T), device="cuda")
    inv = torch.tensor([10000.0 ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64).cuda()
    y = torch.empty(T, C, device="cuda").bfloat16()

    def run():
        y1, _, _ = gb.norm_fwd(h, p["g1"], None, EPS, gb.RMS)
        qkv, _ = gb.norm_linear_fwd(y1, p["wqkv"])
        q, k = qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + HK) * D].view(T, HK, D)
        gb.norm_rope_fwd(q, k, pos, inv, p["gq"], p["gk"], eps=EPS, sections=(8, 12, 12), yq=q, yk=k)
        y.copy_(h)
        gb.norm_linear_fwd(q.reshape(T, H * D), p["wo"], p["bo"], y, "gelu", y=y)  # in place
        return gb.norm_linear_bwd(dout, q.reshape(T, H * D), p["wo"], y, "silu")

    first = [t.clone() for t in (*run(), y)]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = run()
    gr.replay()
    torch.cuda.synchronize()
    for a, b in zip((*outs, y), first):
        assert torch.equal(a, b)
    h.mul_(-2)
    pos.add_(1)
    gr.replay()
    got = [t.clone() for t in (*outs, y)]
    for a, b in zip(got, (*run(), y)):
        assert torch.equal(a, b)
    assert not torch.equal(got[3], first[3])
