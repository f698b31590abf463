"""Outputs that the native binding allocates: the statistics (and the
parameter gradients) of a call share one allocation, up to 1 MB with the main
output, as tensors of their own that behave like any other."""
import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

pytestmark = pytest.mark.gpu


def test_shared_allocations_are_ordinary_tensors():
    for B, C, G in ((1, 8, 1), (3, 40, 4), (7, 520, 65)):
        x = torch.randn(B, 5, C, device="cuda")
        g, b = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
        y, rstd, mean = gb.norm_group_fwd(x, g, b, G)
        dx, dg, db = gb.norm_group_bwd(x, x, g, b, rstd, mean, G)
        for u, v in ((rstd, mean), (dg, db)):
            assert u.is_contiguous() and v.is_contiguous() and u.dtype == v.dtype == torch.float32
            assert u.data_ptr() % 256 == 0 and v.data_ptr() % 256 == 0
            assert u.numel() * 4 <= abs(v.data_ptr() - u.data_ptr())
            keep = v.clone()
            u.fill_(float("nan"))  # writing one leaves the other
            assert torch.equal(v, keep)
            w = v.view(-1).clone().requires_grad_()
            (w * v.view(-1)).sum().backward()
            assert torch.equal(w.grad, v.view(-1))
            del u
            torch.cuda.synchronize()
            assert torch.equal(v, keep)
        assert rstd.shape == mean.shape == (B, G) and dg.shape == db.shape == (C,)


def test_given_and_missing_outputs_mix():
    x = torch.randn(2, 9, 32, device="cuda", dtype=torch.float16)
    g, b = torch.ones_like(x[0, 0]), torch.zeros_like(x[0, 0])
    want = gb.norm_group_fwd(x, g, b, 4, 1e-5, "silu")
    mean = torch.empty(2, 4, device="cuda")
    y = torch.empty_like(x)
    got = gb.norm_group_fwd(x, g, b, 4, 1e-5, "silu", y=y, mean=mean)
    assert got[0].data_ptr() == y.data_ptr() and got[2].data_ptr() == mean.data_ptr()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    full = gb.norm_group_bwd(x, x, g, b, want[1], want[2], 4, "silu")
    part = gb.norm_group_bwd(x, x, g, b, want[1], want[2], 4, "silu", want_dbeta=False)
    assert part[2] is None and torch.equal(part[0], full[0]) and torch.equal(part[1], full[1])


def test_streams_given_as_tensors_streams_and_handles():
    """Outputs and workspaces of a call on another stream belong to that
    stream; results are those of the current one."""
    x = torch.randn(40, 300, 64, device="cuda", dtype=torch.bfloat16)
    g, b = torch.ones_like(x[0, 0]), torch.zeros_like(x[0, 0])
    want = gb.norm_group_fwd(x, g, b, 8, 1e-5, "silu")
    grads = gb.norm_group_bwd(x, x, g, b, want[1], want[2], 8, "silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        for _ in range(3):
            got = gb.norm_group_fwd(x, g, b, 8, 1e-5, "silu", stream=handle)
            back = gb.norm_group_bwd(x, x, g, b, got[1], got[2], 8, "silu", stream=handle)
        s.synchronize()
        for u, v in zip(got + back, want + grads):
            assert torch.equal(u, v)
    assert torch.cuda.current_stream() != s


def test_small_main_outputs_share_with_their_statistics():
    """Up to 1 MB the main output, too, lies in the statistics' allocation:
    none overlaps another, each keeps its values when another is written or
    freed, and a larger output stands alone."""
    for S in (1, 37, 1000, 40000):
        x = torch.randn(2, S, 40, device="cuda", dtype=torch.bfloat16)
        g, b = torch.ones_like(x[0, 0]), torch.zeros_like(x[0, 0])
        y, rstd, mean = gb.norm_group_fwd(x, g, b, 4, 1e-5, "gelu")
        outs = [y, rstd, mean, *gb.norm_group_bwd(x, x, g, b, rstd, mean, 4, "gelu")]
        r2 = x.view(-1, 40)
        outs += gb.norm_dropout_add_fwd(r2, r2, g, b, 1e-5, gb.LAYER, p=0.5, seed=3)
        outs += gb.norm_dropout_add_bwd(r2, r2, outs[6], g, outs[8], outs[9], gb.LAYER, p=0.5, seed=3)
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs)
        assert all(lo % 256 == 0 for lo, _ in spans)
        assert all(hi <= lo for (_, hi), (lo, _) in zip(spans, spans[1:]))
        alone = y.untyped_storage().nbytes() == y.numel() * 2
        assert alone == (y.numel() * 2 > 1 << 20)
        want = [t.clone() for t in outs]
        while outs:
            t, w = outs.pop(0), want.pop(0)
            assert t.is_contiguous() and torch.equal(t, w)
            t.fill_(float("nan"))
            del t
            torch.cuda.synchronize()
        assert torch.isfinite(x).all()
