"""The dropout and group-normalisation entry points without a GPU: refusals
with the documented status codes before CUDA is touched, and the group plans
of a described GB300 (152 SMs, 227 KB of shared memory) in bounds, owning
every row and group once."""
import ctypes

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

F = 16  # a fake, 16-byte aligned address: validation fails before any use
SMS, OPTIN = 152, 232448


def test_dropout_refusals():
    f = gb.lib().norm_dropout
    ok = dict(x=F, n=64, p=0.1, seed=1, off=2, od=None, dt=0, y=F)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["x"], a["n"], a["p"], a["seed"], a["off"], a["od"], a["dt"], a["y"], None)

    assert call(x=None) == 1 and call(y=None) == 1
    assert call(n=0) == 2 and call(n=-1) == 2 and call(n=(1 << 40) + 1) == 2
    assert call(dt=3) == 9 and call(dt=-1) == 9
    for p in (-0.1, 1.0, 2.0, float("nan"), 1 - 2.0 ** -17):
        assert call(p=p) == 9, p
    assert call(x=F + 8) == 3 and call(y=F + 2) == 3 and call(od=F + 4) == 3


def test_dropout_add_refusals():
    f = gb.lib().norm_dropout_add_fwd
    ok = dict(x=F, r=F, g=F, b=None, M=4, N=64, eps=1e-5, mode=0, p=0.1, od=None, h=F, y=F, rs=F,
              m=None)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["x"], a["r"], a["g"], a["b"], a["M"], a["N"], a["eps"], a["mode"], a["p"], 1, 2,
                 a["od"], a["h"], a["y"], a["rs"], a["m"], None)

    for k in ("x", "r", "g", "h", "y", "rs"):
        assert call(**{k: None}) == 1, k
        assert call(**{k: F + 8}) == 3, k
    assert call(N=12) == 2 and call(M=0) == 2 and call(N=262144 + 8) == 2
    assert call(mode=2) == 4 and call(b=F) == 4 and call(m=F) == 4 and call(mode=1) == 4
    assert call(eps=-1.0) == 9 and call(p=1.0) == 9 and call(p=-0.5) == 9 and call(od=F + 4) == 3
    assert call(p=0.0, x=F + 8) == 3

    fb = gb.lib().norm_dropout_add_bwd
    okb = dict(dy=F, dh=F, h=F, g=F, rs=F, m=None, M=4, N=64, mode=0, p=0.1, dx=F, dr=F, dg=F,
              db=None, ws=F, wsb=1 << 20)

    def bwd(**kw):
        a = dict(okb, **kw)
        return fb(a["dy"], a["dh"], a["h"], a["g"], a["rs"], a["m"], a["M"], a["N"], a["mode"],
                 a["p"], 1, 2, None, a["dx"], a["dr"], a["dg"], a["db"], a["ws"], a["wsb"], None)

    for k in ("dy", "dh", "h", "g", "rs", "dx", "dr", "dg"):
        assert bwd(**{k: None}) == 1, k
        assert bwd(**{k: F + 8}) == 3, k
    assert bwd(ws=None) == 5 and bwd(ws=F + 4) == 3
    assert bwd(mode=1) == 4 and bwd(db=F) == 4 and bwd(p=float("inf")) == 9 and bwd(N=20) == 2


def test_group_refusals():
    f = gb.lib().norm_group_fwd
    ok = dict(x=F, g=F, b=F, B=2, S=5, C=32, G=4, eps=1e-5, act=1, dt=0, p=0.0, od=None, y=F, rs=F,
              m=F, ws=None, wsb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["x"], a["g"], a["b"], a["B"], a["S"], a["C"], a["G"], a["eps"], a["act"],
                 a["dt"], a["p"], 1, 2, a["od"], a["y"], a["rs"], a["m"], a["ws"], a["wsb"], None)

    for k in ("x", "g", "y", "rs", "m"):
        assert call(**{k: None}) == 1, k
    for k in ("x", "g", "b", "y", "rs", "m", "ws"):
        assert call(**{k: F + 8}) == 3, k
    for kw in (dict(B=0), dict(S=0), dict(C=0), dict(C=12, G=4), dict(C=8200, G=8), dict(G=0),
               dict(G=5), dict(G=64), dict(B=(1 << 24) + 1), dict(S=(1 << 30) + 1),
               dict(B=1 << 20, S=1 << 21)):
        assert call(**kw) == 2, kw
    for kw in (dict(act=3), dict(act=-1), dict(dt=3), dict(p=1.0), dict(p=-0.1), dict(eps=-1.0),
               dict(eps=float("nan"))):
        assert call(**kw) == 9, kw
    assert call(od=F + 4) == 3
    fb = gb.lib().norm_group_bwd
    okb = dict(dy=F, x=F, g=F, b=None, rs=F, m=F, B=2, S=5, C=32, G=4, act=1, dt=0, p=0.0, dx=F,
              dg=F, db=None, ws=None, wsb=0)

    def bwd(**kw):
        a = dict(okb, **kw)
        return fb(a["dy"], a["x"], a["g"], a["b"], a["rs"], a["m"], a["B"], a["S"], a["C"], a["G"],
                 a["act"], a["dt"], a["p"], 1, 2, None, a["dx"], a["dg"], a["db"], a["ws"],
                 a["wsb"], None)

    for k in ("dy", "x", "g", "rs", "m", "dx", "dg"):
        assert bwd(**{k: None}) == 1, k
        assert bwd(**{k: F + 8}) == 3, k
    assert bwd(db=F + 4) == 3 and bwd(act=7) == 9 and bwd(C=20) == 2 and bwd(p=2.0) == 9
    if not torch.cuda.is_available():
        assert call() == 7 and bwd() == 7  # valid arguments, no device
    n = ctypes.c_size_t(0)
    for q in (gb.lib().norm_group_fwd_workspace_bytes, gb.lib().norm_group_bwd_workspace_bytes):
        assert q(2, 5, 32, 4, 0, None) == 1 and q(2, 5, 32, 3, 0, ctypes.byref(n)) == 2
        assert q(2, 5, 32, 4, 5, ctypes.byref(n)) == 9


def _plan_cases():
    for C, G in ((8, 1), (8, 8), (24, 8), (40, 4), (64, 32), (88, 11), (168, 12), (320, 32),
                 (512, 1), (640, 32), (1280, 32), (2560, 32), (8192, 32), (8192, 8192), (8184, 3)):
        for B in (1, 2, 16, 100, 5000):
            for S in (1, 2, 7, 64, 221, 1024, 4096, 65536, 1 << 20):
                yield B, S, C, G


@pytest.mark.parametrize("override", ["", "form=0", "form=1", "form=1,splits=7", "form=0,k=8",
                                      "form=0,R=2", "form=2", "form=2,R=1,stages=3",
                                      "form=2,nsamp=2,splits=5"])
def test_group_plans_in_bounds(override, monkeypatch):
    if override:
        monkeypatch.setenv("GBNORM_GROUP", override)
    seen = set()
    for B, S, C, G in _plan_cases():
        for dt in (0, 2):
            for bwd in (False, True):
                try:
                    p = gb.norm_group_plan(B, S, C, G, dt, bwd, SMS, OPTIN)
                except gb.NormError as e:
                    assert e.status == 6 and override[:6] in ("form=0", "form=2")
                    continue
                V, D, nt = (4 if dt == 2 else 8), C // G, 2 if bwd else 1
                label = (B, S, C, G, dt, bwd, p)
                seen.add(p["form"])
                R, ncs = p["row_lanes"], p["chunk_columns"]
                assert p["threads"] % 32 == 0 and 32 <= p["threads"] <= 512, label
                assert ncs * R <= p["threads"], label
                assert 0 < p["smem_bytes"] <= OPTIN and 1 <= p["grid"] < 1 << 31, label
                fold = ((R + 1) // 2 * ncs * (8 * V + 4) if R > 1 else 0) + ncs * V * 8
                if p["form"] == 1:
                    assert p["grid"] == B * p["row_splits"] and p["row_splits"] <= max(S, 1), label
                    assert p["smem_bytes"] >= 8 * C + fold - ncs * V * 8, label
                    need = (p["grid"] * G * 8 + 15) // 16 * 16 + (p["grid"] * C * 8 if bwd else 0)
                    if bwd and p["grid"] == 1:
                        need -= C * 8
                    assert p["workspace_bytes"] == need, label
                    continue
                # slabs: whole groups, 16-byte borders, covering every group once
                assert p["groups_per_slab"] * D == ncs * V, label
                assert p["groups_per_slab"] * D % 8 == 0, label
                assert (p["slabs"] - 1) * p["groups_per_slab"] < G <= \
                    p["slabs"] * p["groups_per_slab"], label
                if p["form"] == 2:
                    # one CTA per SM, all resident; every sample in one round;
                    # no CTA with fewer tiles than stages when the ring goes on
                    n, sp, TR = p["samples_per_round"], p["row_splits"], (4 if bwd else 8) * R
                    assert p["grid"] == n * p["slabs"] * sp <= SMS, label
                    assert (p["rounds"] - 1) * n < B <= p["rounds"] * n and sp <= S, label
                    assert 1 <= p["stages"] <= 31, label
                    assert 0 <= p["tensor_memory_tiles"] <= max(0, min(4, -(-(-(-S // sp)) // TR) - p["stages"]))
                    if p["rounds"] > 1:
                        assert -(-(S // sp) // TR) >= p["stages"], label
                    stage = TR * ncs * 16 * nt
                    assert p["smem_bytes"] >= p["stages"] * stage + fold + \
                        (ncs * V * 8 if bwd else 0) + 8 * p["groups_per_slab"] + \
                        16 * p["stages"] + 8, label
                    if bwd:  # the column sums' float per thread before the channel arrays
                        assert p["smem_bytes"] >= p["stages"] * stage + 2048 + 16 * ncs * V
                    if p["tensor_memory_tiles"]:  # never two CTAs on one SM
                        assert 2 * (p["smem_bytes"] + 1024) > OPTIN + 1024, label
                    assert stage < 1 << 20, label  # bytes one stage barrier counts
                    assert p["workspace_bytes"] == (B * G * (sp + sp % 2) * 8) + \
                        (n * sp * C * 8 if bwd else 0), label
                    continue
                assert p["grid"] == B * p["slabs"] * p["cluster"], label
                assert p["cluster"] in (1, 2, 4, 8) and p["cluster"] <= S, label
                assert p["cluster_samples"] in (1, B) and (bwd or p["cluster_samples"] == 1)
                assert p["cluster"] * p["cluster_samples"] <= 8, label
                # rows: every CTA's range fits its threads' slots, and no row
                # lane is empty
                rows = [S * (i + 1) // p["cluster"] - S * i // p["cluster"]
                        for i in range(p["cluster"])]
                assert sum(rows) == S and max(rows) <= p["rows_per_thread"] * R, label
                assert R <= min(rows), label
                data = p["rows_per_thread"] * ncs * R * 16 * nt
                assert p["smem_bytes"] >= data + fold + 16 * p["groups_per_slab"], label
                assert p["workspace_bytes"] == (
                    B * C * 8 if bwd and B > p["cluster_samples"] else 0), label
    assert seen == ({0, 1, 2} if not override else {int(override[5])})


@pytest.mark.parametrize("text", ["R=-3", "stages=-1,form=2", "splits=-2,form=2", "k=-1", "junk"])
def test_shape_override_ignores_negative_values(text, monkeypatch):
    form = ["form=2"] if "form=2" in text else []
    monkeypatch.setenv("GBNORM_GROUP", ",".join(form))
    for back in (False, True):
        want = gb.norm_group_plan(4, 300, 320, 32, gb.BF16, back, SMS, OPTIN)
        monkeypatch.setenv("GBNORM_GROUP", text)
        assert gb.norm_group_plan(4, 300, 320, 32, gb.BF16, back, SMS, OPTIN) == want
        monkeypatch.setenv("GBNORM_GROUP", ",".join(form))


def test_ring_with_tensor_memory_has_its_sm_alone():
    # a CTA that holds all of an SM's tensor memory while it waits for its peers
    # leaves no shared memory for one that would wait for that tensor memory
    seen = 0
    for B, S, C, G in ((1, 262144, 256, 32), (4, 16384, 512, 32), (16, 4096, 320, 32),
                       (64, 1024, 640, 32), (3, 9000, 64, 8), (300, 2048, 1280, 32)):
        for dtype in (gb.BF16, gb.FP16, gb.FP32):
            for back in (False, True):
                p = gb.norm_group_plan(B, S, C, G, dtype, back, SMS, OPTIN)
                if p["form"] == 2 and p["tensor_memory_tiles"]:
                    seen += 1
                    assert p["smem_bytes"] == OPTIN, (B, S, C, dtype, back)
    assert seen >= 6
