"""Forced forms of the linear layer's gradients (GBNORM_LINEAR): tile widths, cluster
sizes, one launch for both products or one each, at ragged sizes."""
import pytest
import torch

import linear_ref as lr
import memory_bound_normalization_rmsnorm_gb300 as gb
from test_linear import FORMS, _bwd_check, _make
from test_linear_sums import backward_limits, check_rms

SIZES = [(5, 70, 33), (300, 600, 328), (130, 64, 264), (257, 520, 513), (640, 200, 1000)]


def _check(c, name):
    z = lr.forward(c["x"], c["w"], c["bias"], None, name)[0][1].to(c["x"].dtype)
    want, most = backward_limits(c["dy"], c["x"], c["w"], z, name)
    zin = z if name != "none" else None
    calls = [{}, dict(want_dw=False), dict(want_dx=False), dict(want_dbias=False),
             dict(want_dw=False, want_dbias=False), dict(want_dx=False, want_dbias=False)]
    for kw in calls:
        got = gb.norm_linear_bwd(c["dy"], c["x"], c["w"], zin, name, **kw)
        _bwd_check(c, name, got)
        for n, g, w, m in zip(("dx", "dw", "dbias"), got, want, most):
            assert (g is None) == (f"want_{n}" in kw)
            if g is not None:
                check_rms(g, w, m, n)


@pytest.mark.gpu
@pytest.mark.parametrize("joint", [0, 1])
@pytest.mark.parametrize("form", [f for f in FORMS if f.startswith("pair=0")])
def test_split_gradients(form, joint, monkeypatch):
    monkeypatch.setenv("GBNORM_LINEAR", f"{form},joint={joint}")
    for shape in SIZES:
        for dtype, name in (("bf16", "none"), ("fp16", "gelu")):
            _check(_make(dtype, *shape), name)
    assert gb.norm_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("form", [f for f in FORMS if f.startswith("pair=1")])
def test_pair_gradients(form, monkeypatch):
    monkeypatch.setenv("GBNORM_LINEAR", form)
    for shape in SIZES:
        _check(_make("bf16", *shape), "silu")
    assert gb.norm_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("joint", [0, 1])
def test_forced_cluster_sizes_reach_the_gradients(joint, monkeypatch):
    """Another cut of the contraction rounds other partial sums: of 100 000 fp16 outputs
    and more over 1024 and 256 terms some differ in their last place."""
    c = _make("fp16", 256, 512, 1024)
    got = {}
    for splits in (1, 2, 4):
        monkeypatch.setenv("GBNORM_LINEAR", f"pair=0,bn=64,splits={splits},joint={joint}")
        got[splits] = gb.norm_linear_bwd(c["dy"], c["x"], c["w"])
        _bwd_check(c, "none", got[splits])
    for a, b in ((1, 2), (2, 4), (1, 4)):
        for i in (0, 1):
            assert not torch.equal(got[a][i], got[b][i])


@pytest.mark.gpu
def test_one_launch_or_two_by_the_environment(monkeypatch):
    """The bias sum behind joint products adds the partial rows (128 here) one after
    the other, the kernel of its own 32 side by side: other bits, both within bounds."""
    c = _make("bf16", 4096, 64, 256)
    got = []
    for joint in (0, 1):
        monkeypatch.setenv("GBNORM_LINEAR", f"pair=0,joint={joint}")
        got.append(gb.norm_linear_bwd(c["dy"], c["x"], c["w"]))
        _bwd_check(c, "none", got[-1])
    assert not torch.equal(got[0][2], got[1][2])
