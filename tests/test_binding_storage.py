"""Every new output of the native binding owns its memory: releasing or
growing one (as sharding and offloading code does to activations) leaves the
others, which a backward pass may still need."""
import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

pytestmark = pytest.mark.gpu

RNG = dict(p=0.25, seed=7, offset=3)


def _group(S=37):
    gen = torch.Generator().manual_seed(S)
    x, dy = (torch.randn(2, S, 40, generator=gen).bfloat16().cuda() for _ in range(2))
    g, b = torch.ones(40, device="cuda", dtype=x.dtype), torch.zeros(40, device="cuda",
                                                                     dtype=x.dtype)
    return x, dy, g, b


def _outputs(S):
    x, dy, g, b = _group(S)
    rows, drows = x.view(-1, 40), dy.view(-1, 40)
    fwd = gb.norm_group_fwd(x, g, b, 4, 1e-5, "silu", **RNG)
    bwd = gb.norm_group_bwd(dy, x, g, b, fwd[1], fwd[2], 4, "silu", **RNG)
    add = gb.norm_dropout_add_fwd(rows, drows, g, b, 1e-5, gb.LAYER, **RNG)
    back = gb.norm_dropout_add_bwd(drows, rows, add[0], g, add[2], add[3], gb.LAYER, **RNG)
    return [*fwd, *bwd, *add, *back, gb.norm_dropout(x, **RNG)]


def _own(outs):
    """Asserts that no two share a storage (before anything is released)."""
    at = [t.untyped_storage().data_ptr() for t in outs]
    assert len(set(at)) == len(at), "two outputs share a storage"
    for t in outs:
        assert t.storage_offset() == 0
        assert 0 <= t.untyped_storage().nbytes() - t.numel() * t.element_size() < 512


@pytest.mark.parametrize("S", [1, 37, 4000])
def test_each_output_owns_its_storage(S):
    _own(_outputs(S))


@pytest.mark.parametrize("S", [1, 37, 4000])
def test_releasing_one_storage_leaves_the_others(S):
    for i in range(len(_outputs(S))):
        outs = _outputs(S)
        _own(outs)
        want = [t.clone() for t in outs]
        freed = outs[i].untyped_storage().nbytes()
        outs[i].untyped_storage().resize_(0)
        # whatever takes the memory next must not show in the others
        fill = [torch.full((freed,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        for j, (t, w) in enumerate(zip(outs, want)):
            assert j == i or torch.equal(t, w), (i, j)
        del fill


@pytest.mark.parametrize("S", [1, 37, 4000])
def test_growing_one_output_leaves_the_others(S):
    for i in range(len(_outputs(S))):
        outs = _outputs(S)
        _own(outs)
        want = [t.clone() for t in outs]
        outs[i].resize_(outs[i].numel() + 700).fill_(float("nan"))
        for j, (t, w) in enumerate(zip(outs, want)):
            assert j == i or torch.equal(t, w), (i, j)


def test_backward_after_the_activation_was_released():
    x, dy, g, b = _group()
    y, rstd, mean = gb.norm_group_fwd(x, g, b, 4, 1e-5, "silu")
    want = gb.norm_group_bwd(dy, x, g, b, rstd, mean, 4, "silu")
    _own([y, rstd, mean])
    y.untyped_storage().resize_(0)
    torch.full((1 << 16,), float("nan"), device="cuda")
    got = gb.norm_group_bwd(dy, x, g, b, rstd, mean, 4, "silu")
    for u, v in zip(got, want):
        assert torch.equal(u, v)


def test_recorded_streams_hold_an_output():
    """record_stream keeps each output's memory from being given out again
    while the other stream may still read it."""
    s = torch.cuda.Stream()
    for i in range(len(_outputs(37))):
        outs = _outputs(37)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        n, at = outs[i].untyped_storage().nbytes(), outs[i].data_ptr()
        outs[i].record_stream(s)
        outs[i] = None
        later = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert at not in [t.data_ptr() for t in later]
        torch.cuda.synchronize()
