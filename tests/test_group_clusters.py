"""The backward's exchange over a cluster without dbeta: only sums that are
stored are read from the peers (one whose value nothing waits for could still
be on its way when the peer leaves), and dx and dgamma are those of a call with
dbeta, in every cluster shape."""
import os
import re

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

CSRC = os.path.join(os.path.dirname(gb.__file__), "csrc")


def test_every_remote_read_is_conditional_on_its_store():
    """In the source: the peers' sums for dbeta are read, and stored, under the
    same condition."""
    with open(os.path.join(CSRC, "group_bwd.cu")) as f:
        text = f.read()
    assert "const bool want_b = a.dbeta_part != nullptr;" in text
    branch = re.search(r"\} else if \(want_b\) \{\n(.*?)\n    \} else \{\n", text, re.S)
    assert branch and branch.group(1).count("ld_cluster_f2(pb, ") == 1
    assert text.count("ld_cluster_f2(pb, ") == 1
    stores = re.findall(r"^.*a\.dbeta_part \+ at\) = tb.*$", text, re.M)
    assert len(stores) == 1 and stores[0].strip().startswith("if (want_b) ")


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 2, 4, 8])
@pytest.mark.parametrize("B", [1, 2, 3, 7, 8, 20])
def test_without_dbeta_over_clusters(B, k, monkeypatch):
    gen = torch.Generator().manual_seed(10 * B + k)
    for S, C, G in ((8, 64, 8), (50, 320, 32)):
        x, dy = (torch.randn(B, S, C, generator=gen).bfloat16().cuda() for _ in range(2))
        g, b = (torch.randn(C, generator=gen).bfloat16().cuda() for _ in range(2))
        for cb in ("", ",cb=1"):
            monkeypatch.setenv("GBNORM_GROUP", f"form=0,k={k}{cb}")
            _, rstd, mean = gb.norm_group_fwd(x, g, b, G, 1e-5, "silu")
            full = gb.norm_group_bwd(dy, x, g, b, rstd, mean, G, "silu")
            for _ in range(20):
                part = gb.norm_group_bwd(dy, x, g, b, rstd, mean, G, "silu", want_dbeta=False)
                assert part[2] is None
                assert torch.equal(part[0], full[0]) and torch.equal(part[1], full[1])
    assert gb.norm_get_device_error() == 0
