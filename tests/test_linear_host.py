"""Host side of the linear layer, without a GPU."""
import ctypes
import os
import re

import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

CSRC = os.path.join(os.path.dirname(gb.__file__), "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_every_launch_carries_the_error_word():
    """A wait that runs out sets a bit of the device's error word: each argument
    structure that has its address gets it wherever one is made."""
    header, text = _source("linear.cuh"), _source("linear.cu")
    with_err = [m.group(1) for m in re.finditer(r"struct (\w+) \{(?:(?!\n\};).)*unsigned \*err;", header, re.S)]
    assert sorted(with_err) == ["PairArgs", "SplitArgs"]
    made = re.findall(r"\b(?:PairArgs|SplitArgs) (\w+) = \{\};", text)
    assert sorted(made) == ["args", "p"]
    for name in made:
        assert len(re.findall(rf"\b{name}\.err = d\.err;", text)) == 1
    # the split form's are made in the constructor of a launch, its only one
    assert re.findall(r"^  (?:explicit )?SplitLaunch\((.*?)\)", text, re.M) == ["const Device &d, int splits"]


def test_backward_query_refuses_what_the_call_refuses():
    """norm_linear_bwd_workspace_bytes: strides and addresses, as the forward's query."""
    F, n = 256, ctypes.c_size_t(7)
    ok = dict(dy=F, lddy=32, x=F, ldx=64, w=F, ldw=64, z=F, ldz=32, dx=1, dw=1)

    def query(**kw):
        a = dict(ok, **kw)
        return gb.lib().norm_linear_bwd_workspace_bytes(
            a["dy"], a["lddy"], a["x"], a["ldx"], a["w"], a["ldw"], a["z"], a["ldz"], 4, 64, 32, 1,
            a["dx"], a["dw"], 1, ctypes.byref(n))

    for kw in (dict(lddy=31), dict(ldx=63), dict(ldw=0), dict(ldz=-32), dict(ldx=(1 << 32) + 8)):
        assert query(**kw) == 2
    for kw in (dict(dy=F + 1), dict(x=F + 1), dict(w=F + 1), dict(z=F + 1)):
        assert query(**kw) == 3
    if not torch.cuda.is_available():
        assert query() == 7
        # what is not read is not looked at
        assert query(w=None, ldw=0, dx=0) == 7 and query(x=F + 1, ldx=0, dw=0) == 7
