"""Host side of the linear layer, without a GPU."""
import os
import re

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
