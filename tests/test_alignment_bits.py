"""What the bits of the linear layer's and the rotation's results depend on: shape,
type and alignment, not the address itself."""
import pytest
import torch

import linear_ref as lr
import memory_bound_normalization_rmsnorm_gb300 as gb


def _at(t, offset, pad):
    """The values of t [M, C] `offset` elements into a buffer of rows C + pad."""
    flat = torch.zeros(t.shape[0] * (t.shape[1] + pad) + offset, device="cuda", dtype=t.dtype)
    rows = flat[offset:].view(t.shape[0], -1)[:, :t.shape[1]]
    rows.copy_(t)
    return rows


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(300, 256, 520), (2304, 136, 1544)])
def test_linear(shape):
    M, K, N = shape
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, dy, z = rnd(M, K), rnd(N, K) / 16, rnd(M, N), rnd(M, N)
    y, _ = gb.norm_linear_fwd(x, w, None, z, "gelu")
    want = gb.norm_linear_bwd(dy, x, w, z, "gelu")
    db64 = lr.backward(dy, x, w, z, "gelu")
    for offset, pad in ((8, 0), (64, 24), (1, 3), (2, 1)):
        mx, mw, mdy, mz = (_at(t, offset, pad) for t in (x, w, dy, z))
        assert torch.equal(gb.norm_linear_fwd(mx, mw, None, mz, "gelu")[0], y)
        dx, dw, db = gb.norm_linear_bwd(mdy, mx, mw, mz, "gelu")
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        if offset % 8 == 0:
            assert torch.equal(db, want[2])
        lr.check(db, db64[0][2], db64[1][2], "dbias")


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_rotation(inter):
    g = torch.Generator(device="cuda").manual_seed(2)
    T, H, D = 37, 6, 128
    q, dy = (torch.randn(T, H * D, generator=g, device="cuda").bfloat16() for _ in range(2))
    gamma = torch.randn(D, generator=g, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda") * 1000
    inv = torch.tensor([0.8 ** i for i in range(D // 2)], device="cuda", dtype=torch.float64)
    first = None
    for offset, pad in ((0, 0), (8, 0), (64, 24)):
        mq, mdy = (_at(t, offset, pad).unflatten(1, (H, D)) for t in (q, dy))
        got = [gb.norm_rope_fwd(mq, None, pos, inv, gamma, interleaved=inter)[0]]
        dq, _, dgamma, _, _, _ = gb.norm_rope_bwd(mdy, None, mq, None, pos, inv, gamma, interleaved=inter)
        got += [dq, dgamma]
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b)
