"""norm_group_fwd / norm_group_bwd against the float64 definitions, in both
forms (resident and streamed) and every way a resident unit is split."""
import ctypes

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

import dropout_ref as dref
import group_ref as ref

pytestmark = pytest.mark.gpu

SEED, OFF = 0xD1B54A32D192ED03, (9 << 32) + 2
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(B, S, C, dtype, seed=0, shift=0.5, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (scale * (r(B, S, C) + shift * r(C))).to(dtype)
    return [t.cuda() for t in (x, (1 + 0.2 * r(C)).to(dtype), (0.2 * r(C)).to(dtype),
                               r(B, S, C).to(dtype))]


def factor(x, p):
    if not p:
        return None
    k = dref.keep(tuple(x.shape), p, SEED, OFF).to(x.device).double()
    return k * (65536.0 / (65536 - dref.threshold(p)))


def check_both(x, gamma, beta, dy, G, act, p, label, eps=1e-5):
    rng = dict(p=p, seed=SEED, offset=OFF)
    y, rstd, mean = gb.norm_group_fwd(x, gamma, beta, G, eps, act, **rng)
    dx, dg, db = gb.norm_group_bwd(dy, x, gamma, beta, rstd, mean, G, act, **rng)
    torch.cuda.synchronize()
    B, C = x.shape[0], x.shape[-1]
    x3, dy3 = x.reshape(B, -1, C), dy.reshape(B, -1, C)
    fac = factor(x3, p)
    y64, r64, m64, mag = ref.forward(x3, gamma, beta, G, eps, act, fac)
    ref.check(y.reshape(x3.shape), y64, mag, f"{label} y")
    # statistics: relative to their own terms
    sd = 1 / r64
    ref.check(mean, m64, m64.abs() + sd, f"{label} mean")
    ref.check(rstd, r64, r64 * (1 + (m64 * r64).abs()), f"{label} rstd")
    want = ref.backward(dy3, x3, gamma, beta, rstd, mean, G, act, fac)
    for got, w, m, n in zip((dx.reshape(x3.shape), dg, db), want[:3], want[3:],
                            ("dx", "dgamma", "dbeta")):
        ref.check(got, w, m, f"{label} {n}")
    return y, rstd, mean, dx, dg, db


# one position, one channel per group, groups across chunk borders (10, 14, 3
# channels), whole-sample groups, one group per channel, more chunk columns
# than a CTA has threads, ragged positions, many small samples
SHAPES = [(1, 1, 8, 1), (1, 1, 8, 8), (2, 1, 64, 4), (2, 7, 16, 2), (3, 64, 40, 4),
          (1, 257, 24, 8), (2, 100, 320, 32), (5, 33, 168, 12), (1, 2048, 64, 32),
          (2, 1024, 512, 1), (1, 70, 8192, 32), (1, 2, 8192, 8192), (40, 9, 64, 8),
          (2, 221, 88, 11), (1, 64, 1280, 32), (3, 1517, 168, 12), (700, 3, 64, 8)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_parity(shape, dtype):
    B, S, C, G = shape
    x, g, b, dy = make(B, S, C, DT[dtype], seed=B + S + C)
    for act in ("none", "silu", "gelu"):
        check_both(x, g, b, dy, G, act, 0.0, f"{shape} {dtype} {act}")
    check_both(x, g, b, dy, G, "silu", 0.1, f"{shape} {dtype} silu p=0.1")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] > 1], ids=str)
def test_parity_streamed(shape, dtype, monkeypatch):
    B, S, C, G = shape
    x, g, b, dy = make(B, S, C, DT[dtype], seed=B + S + C + 1)
    for splits in ("", ",splits=1", ",splits=3", ",splits=5"):
        monkeypatch.setenv("GBNORM_GROUP", "form=1" + splits)
        plan = gb.norm_group_plan(B, S, C, G, ["bf16", "fp16", "fp32"].index(dtype))
        assert plan["form"] == 1
        check_both(x, g, b, dy, G, "gelu", 0.25, f"{shape} {dtype} streamed{splits}")
        check_both(x, g, None, dy, G, "none", 0.0, f"{shape} {dtype} streamed{splits} no beta")


RINGS = ["", ",R=1", ",splits=1,R=1,stages=3", ",splits=2,R=2,stages=2", ",splits=3,R=1,stages=4",
         ",nsamp=1,splits=1,R=1,stages=2", ",nsamp=1,splits=2,R=1", ",nsamp=2,splits=1,R=2,stages=3",
         ",splits=1,R=1,stages=2,tm=0", ",splits=1,R=1,stages=1,tm=2"]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [s for s in SHAPES if s != (1, 2, 8192, 8192)], ids=str)
def test_parity_ring(shape, dtype, monkeypatch):
    """One tile, fewer tiles than stages, many turns of the ring, several
    rounds (a last one with fewer samples), row ranges of unequal length."""
    B, S, C, G = shape
    x, g, b, dy = make(B, S, C, DT[dtype], seed=B + S + C + 2)
    for ring in RINGS:
        monkeypatch.setenv("GBNORM_GROUP", "form=2" + ring)
        assert gb.norm_group_plan(B, S, C, G, list(DT).index(dtype))["form"] == 2
        check_both(x, g, b, dy, G, "silu", 0.1, f"{shape} {dtype} ring{ring}")
        check_both(x, g, None, dy, G, "none", 0.0, f"{shape} {dtype} ring{ring} no beta")
    assert gb.norm_get_device_error() == 0


@pytest.mark.parametrize("shape,sg", [((2, 100, 320, 32), 12), ((5, 33, 168, 12), 8),
                                      ((3, 64, 40, 4), 4), ((2, 221, 88, 11), 4)], ids=str)
def test_parity_ring_slabs(shape, sg, monkeypatch):
    """Slabs narrower than a row (copied row by row), the last one narrower."""
    B, S, C, G = shape
    for dtype in DT.values():
        x, g, b, dy = make(B, S, C, dtype, seed=sg)
        for ring in RINGS[:5]:
            monkeypatch.setenv("GBNORM_GROUP", f"form=2,sg={sg}" + ring)
            check_both(x, g, b, dy, G, "gelu", 0.1, f"{shape} sg={sg} ring{ring}")
    assert gb.norm_get_device_error() == 0


@pytest.mark.parametrize("k", [1, 2, 4, 8])
@pytest.mark.parametrize("shape,sg", [((2, 100, 320, 32), 4), ((2, 100, 320, 32), 12),
                                      ((5, 33, 168, 12), 12), ((3, 64, 40, 4), 4),
                                      ((1, 257, 24, 8), 8), ((2, 8, 64, 8), 1),
                                      ((2, 221, 88, 11), 4)], ids=str)
def test_parity_resident_splits(shape, sg, k, monkeypatch):
    """Every cluster size, slabs narrower than the last one, one row lane."""
    B, S, C, G = shape
    x, g, b, dy = make(B, S, C, torch.bfloat16, seed=k)
    for R in ("", ",R=1", ",R=3", ",cb=1"):
        monkeypatch.setenv("GBNORM_GROUP", f"form=0,sg={sg},k={k}{R}")
        plan = gb.norm_group_plan(B, S, C, G)
        assert plan["form"] == 0 and plan["cluster"] == k
        check_both(x, g, b, dy, G, "silu", 0.1, f"{shape} sg={sg} k={k}{R}")


@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("B", [1, 3, 9, 40])
def test_gradients_without_dbeta(B, form, monkeypatch):
    """dbeta left out, for one partial row, a batch in a cluster and more."""
    monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
    x, g, b, dy = make(B, 30, 64, torch.bfloat16, seed=B)
    y, rstd, mean = gb.norm_group_fwd(x, g, b, 8, 1e-5, "silu")
    full = gb.norm_group_bwd(dy, x, g, b, rstd, mean, 8, "silu")
    part = gb.norm_group_bwd(dy, x, g, b, rstd, mean, 8, "silu", want_dbeta=False)
    assert part[2] is None
    assert torch.equal(part[0], full[0]) and torch.equal(part[1], full[1])


def test_two_calls_at_once():
    """Calls on two streams, each with workspaces of its own, resident and
    whole-GPU forms side by side."""
    big = make(1, 60000, 256, torch.bfloat16, seed=1)
    small = make(20, 300, 64, torch.bfloat16, seed=2)

    def step(case, G):
        x, g, b, dy = case
        y, rstd, mean = gb.norm_group_fwd(x, g, b, G, 1e-5, "silu")
        return (y, rstd, mean, *gb.norm_group_bwd(dy, x, g, b, rstd, mean, G, "silu"))

    want = [step(big, 32), step(small, 8)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s, (case, G) in zip(streams, ((big, 32), (small, 8), (big, 32))):
            with torch.cuda.stream(s):
                got.append(step(case, G))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for u, v in zip(g, want[1 if i % 3 == 1 else 0]):
            assert torch.equal(u, v)
    assert gb.norm_get_device_error() == 0


@pytest.mark.parametrize("form", [0, 1, 2])
def test_statistics_far_from_the_origin(form, monkeypatch):
    """Mean 1000 times the deviation, and a sample whose first rows are zero:
    a sum of squares about the origin would lose every digit of the variance."""
    monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
    x, g, b, dy = make(2, 300, 64, torch.float32, seed=4)
    x = x + 1000.0
    x[1, :40] = 0.0
    check_both(x, g, b, dy, 4, "none", 0.0, "offset")
    y, rstd, mean = gb.norm_group_fwd(x, g, b, 4, 1e-5, "none")
    _, r64 = ref.stats(x, 4, 1e-5)
    assert ((rstd.double() - r64).abs() / r64).max() < 1e-3


def test_constant_groups_and_eps():
    """Zero variance: rstd is 1 / sqrt(eps), y is act(beta)."""
    x, g, b, dy = make(2, 50, 32, torch.float32)
    x.fill_(3.0)
    y, rstd, mean = gb.norm_group_fwd(x, g, b, 4, 1e-4, "silu")
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-5)
    assert torch.equal(mean, torch.full_like(mean, 3.0))
    assert torch.allclose(y, torch.nn.functional.silu(b).expand_as(y), rtol=1e-5, atol=1e-7)


@pytest.mark.parametrize("form", [0, 1, 2])
def test_nan_and_infinity_stay_in_their_group(form, monkeypatch):
    monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
    x, g, b, dy = make(3, 40, 40, torch.bfloat16)
    clean = gb.norm_group_fwd(x, g, b, 4, 1e-5, "silu")
    x2 = x.clone()
    x2[1, 7, 13] = float("nan")   # group 1 (channels 10 to 19), straddles a chunk
    x2[2, 0, 35] = float("inf")   # group 3
    y, rstd, mean = gb.norm_group_fwd(x2, g, b, 4, 1e-5, "silu")
    hit = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[2, 3] = True
    assert torch.equal(torch.isnan(rstd), hit)
    hy = hit[:, None, :, None].expand(3, 40, 4, 10).reshape(3, 40, 40)
    assert torch.isnan(y[hy]).all() and torch.equal(y[~hy], clean[0][~hy])


def test_large_activations_have_finite_gradients():
    """|z| up to 1e15 and beyond: the sigmoid saturates, z k'(z) overflows."""
    x, g, b, dy = make(1, 16, 16, torch.float32)
    for name in ("silu", "gelu"):
        for big in (1e3, 1e8, 1e15, 1e25):
            gg = g * big
            y, rstd, mean = gb.norm_group_fwd(x, gg, b, 2, 1e-5, name)
            dx, dg, db = gb.norm_group_bwd(dy, x, gg, b, rstd, mean, 2, name)
            assert all(torch.isfinite(t).all() for t in (y, dg, db)), (name, big)
            y64, _, _, mag = ref.forward(x, gg, b, 2, 1e-5, name)
            ref.check(y, y64, mag, f"{name} {big} y")
            want = ref.backward(dy, x, gg, b, rstd, mean, 2, name)
            ref.check(db, want[2], want[5], f"{name} {big} dbeta")
            ref.check(dg, want[1], want[4], f"{name} {big} dgamma")


def test_determinism_streams_and_graph():
    """Bitwise the same on another stream and from a replayed graph that
    captured forward and backward."""
    for shape in ((2, 600, 320, 32), (1, 40000, 256, 32), (3, 30000, 512, 32)):
        B, S, C, G = shape
        x, g, b, dy = make(B, S, C, torch.bfloat16)
        a = check_both(x, g, b, dy, G, "silu", 0.1, str(shape)) if S < 1000 else None
        rng = dict(p=0.1, seed=SEED, offset=OFF)

        def step():
            y, rstd, mean = gb.norm_group_fwd(x, g, b, G, 1e-5, "silu", **rng)
            return (y, rstd, mean, *gb.norm_group_bwd(dy, x, g, b, rstd, mean, G, "silu", **rng))

        a = a or step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c = step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            d = step()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for u, v, w in zip(a, c, d):
            assert torch.equal(u, v) and torch.equal(u, w)


@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("dtype", list(DT))
def test_guard_bands(dtype, form, monkeypatch):
    """Nothing is written outside the outputs and the stated workspace."""
    monkeypatch.setenv("GBNORM_GROUP", f"form={form}")
    B, S, C, G = 3, 77, 40, 4
    t = DT[dtype]
    x, g, b, dy = make(B, S, C, t)
    code = list(DT).index(dtype)

    def band(shape, dt):
        n = 1
        for v in shape:
            n *= v
        buf = torch.full((n * dt.itemsize + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[4096:4096 + n * dt.itemsize].view(dt).view(shape)

    wf = gb.norm_group_fwd_workspace_bytes(B, S, C, G, code)
    wb = gb.norm_group_bwd_workspace_bytes(B, S, C, G, code)
    f32, u8 = torch.float32, torch.uint8
    bands = [band((B, S, C), t), band((B, G), f32), band((B, G), f32), band((wf,), u8),
             band((B, S, C), t), band((C,), f32), band((C,), f32), band((wb,), u8)]
    v = [w for _, w in bands]
    gb.norm_group_fwd(x, g, b, G, 1e-5, "silu", y=v[0], rstd=v[1], mean=v[2], workspace=v[3])
    gb.norm_group_bwd(dy, x, g, b, v[1], v[2], G, "silu", dx=v[4], dgamma=v[5], dbeta=v[6],
                      workspace=v[7])
    torch.cuda.synchronize()
    for buf, _ in bands:
        assert (buf[:4096] == 0xA5).all() and (buf[-4096:] == 0xA5).all()


def test_offsets_past_31_bits():
    """A sample that starts beyond 2^31 elements: the same result as alone."""
    B, S, C, G = 3, (1 << 20) + 3, 1024, 32
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.randn(B, S, C, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(C, device="cuda", dtype=torch.bfloat16)
    y, rstd, mean = gb.norm_group_fwd(x, g, None, G, 1e-5, "silu")
    y1, rstd1, mean1 = gb.norm_group_fwd(x[2:], g, None, G, 1e-5, "silu")
    # both within u |y| + 2^-16 (|xhat| + 2) of the same value
    assert torch.allclose(rstd[2:], rstd1, rtol=2.0 ** -15)
    m = (x[2:, -4096:].float().abs() * rstd1.max() + 2) * 2.0 ** -15
    a, c = y[2:, -4096:].float(), y1[:, -4096:].float()
    assert ((a - c).abs() <= 2.0 ** -7 * a.abs() + m).all()
    dx, dg, db = gb.norm_group_bwd(x, x, g, None, rstd, mean, G, "silu", dx=y)
    dx1, _, _ = gb.norm_group_bwd(x[2:], x[2:], g, None, rstd1, mean1, G, "silu", dx=y1)
    a, c = dx[2:, -4096:].float(), dx1[:, -4096:].float()
    assert ((a - c).abs() <= 2.0 ** -7 * a.abs() + 4 * m * (x[2:, -4096:].float().abs() + 1)).all()
    del x, y, y1, dx, dx1
    torch.cuda.empty_cache()


def test_residual_block_run():
    """The operators as a convolutional residual block and the transformer
    block behind it use them: group norm + SiLU + dropout on a channels_last
    tensor, its positions as rows of the dropout + residual add + LayerNorm,
    and the gradients back through both, against float64."""
    B, H, W, C, G, p, eps = 2, 12, 9, 64, 8, 0.1, 1e-5
    x, g, b, _ = make(B, H * W, C, torch.bfloat16, seed=8)
    x4 = x.view(B, H, W, C).permute(0, 3, 1, 2)  # [B, C, H, W], channels_last
    assert x4.is_contiguous(memory_format=torch.channels_last)
    xl = x4.permute(0, 2, 3, 1)
    rng = dict(p=p, seed=SEED, offset=OFF)
    y, rstd, mean = gb.norm_group_fwd(xl, g, b, G, eps, "silu", **rng)
    # fused dropout is norm_dropout of the activation, up to its rounding
    y0, _, _ = gb.norm_group_fwd(xl, g, b, G, eps, "silu")
    sep = gb.norm_dropout(y0, p, SEED, OFF)
    assert torch.equal(sep == 0, (y == 0) | (y0 == 0))
    assert ((sep.float() - y.float()).abs() <= 2.0 ** -7 * y.float().abs() * (1 + 2.0 ** -6)).all()
    rows = y.view(-1, C)
    gl, bl = torch.ones(C, device="cuda", dtype=torch.bfloat16), torch.zeros_like(g)
    r2 = dict(p=p, seed=SEED, offset=OFF + 1)
    h, z, rs2, mu2 = gb.norm_dropout_add_fwd(rows, xl.reshape(-1, C), gl, bl, eps, gb.LAYER, **r2)
    dz, dh = torch.randn_like(z), torch.randn_like(z)
    drows, dres, dgl, dbl = gb.norm_dropout_add_bwd(dz, dh, h, gl, rs2, mu2, gb.LAYER, **r2)
    dx, dg, db = gb.norm_group_bwd(drows.view(B, H, W, C), xl, g, b, rstd, mean, G, "silu", **rng)
    # float64, each stage on the tensors that the kernels handed on
    fac2 = dref.keep((B * H * W, C), p, SEED, OFF + 1).cuda().double()
    fac2 = fac2 * (65536.0 / (65536 - dref.threshold(p)))
    h64 = xl.reshape(-1, C).double() + rows.double() * fac2
    assert ((h.double() - h64).abs() <= 2.0 ** -8 * h64.abs() * (1 + 2.0 ** -15) + 2.0 ** -20).all()
    leaf = h.double().requires_grad_()
    out = torch.nn.functional.layer_norm(leaf, (C,), gl.double(), bl.double(), eps)
    assert ((z.double() - out).abs() <= 2.0 ** -8 * out.abs() + 2.0 ** -16 * 8).all()
    t, = torch.autograd.grad(out, leaf, dz.double())
    t = t + dh.double()
    lim = 2.0 ** -16 * 8 * (1 + t.abs().max())
    assert ((dres.double() - t).abs() <= 2.0 ** -8 * t.abs() + lim).all()
    assert ((drows.double() - t * fac2).abs() <= 2.0 ** -8 * (t * fac2).abs() + 2 * lim).all()
    x3 = x.view(B, H * W, C)
    want = ref.backward(drows.view(x3.shape), x3, g, b, rstd, mean, G, "silu", factor(x3, p))
    ref.check(dx.reshape(x3.shape), want[0], want[3], "block dx")
    ref.check(dg, want[1], want[4], "block dgamma")
    ref.check(db, want[2], want[5], "block dbeta")
    assert gb.norm_get_device_error() == 0


def test_binding_refuses():
    x, g, b, dy = make(2, 8, 32, torch.bfloat16)
    with pytest.raises(ValueError):
        gb.norm_group_fwd(x.transpose(0, 1), g, b, 4)           # strides
    with pytest.raises(ValueError):
        gb.norm_group_fwd(x, g.float(), b, 4)                   # type of gamma
    with pytest.raises(ValueError):
        gb.norm_group_fwd(x.double(), g, b, 4)
    with pytest.raises(ValueError):
        gb.norm_group_fwd(x, g, b, 4, act="relu")
    with pytest.raises(ValueError):
        gb.norm_group_fwd(x, g, b, 4, offset_dev=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(gb.NormError) as e:
        gb.norm_group_fwd(x, g, b, 5)                           # 32 % 5
    assert e.value.status == 2
    with pytest.raises(gb.NormError) as e:
        gb.norm_group_fwd(x, g, b, 4, p=1.0)
    assert e.value.status == 9
    with pytest.raises(gb.NormError) as e:
        many = x.repeat(10, 1, 1)  # a batch that one cluster does not hold
        gb.norm_group_bwd(many, many, g, b, torch.ones(20, 4, device="cuda"),
                          torch.zeros(20, 4, device="cuda"), 4,
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    with pytest.raises(gb.NormError) as e:
        gb.norm_group_fwd(x.view(-1)[4:4 + 32 * 8].view(1, 8, 32), g, b, 4)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        gb.norm_dropout(x.cpu(), 0.1, 1)
    with pytest.raises(ValueError):
        gb.norm_dropout(x, 0.1, -1)
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_binding_refuses_counts_and_codes_out_of_range():
    # refused by value, before an output of that size is asked for
    x, g, b, dy = make(2, 8, 32, torch.bfloat16)
    one = torch.ones(2, 4, device="cuda")
    for groups in (0, -4, 33, 1 << 40):
        with pytest.raises(gb.NormError) as e:
            gb.norm_group_fwd(x, g, b, groups)
        assert e.value.status == 2, groups
        with pytest.raises(gb.NormError) as e:
            gb.norm_group_bwd(dy, x, g, b, one, one, groups)
        assert e.value.status == 2, groups
    for act in (3, -1, 1 << 32):
        with pytest.raises(gb.NormError) as e:
            gb.norm_group_fwd(x, g, b, 4, act=act)
        assert e.value.status == 9, act
    with pytest.raises(gb.NormError) as e:
        gb.norm_dropout_add_fwd(x, x, g, mode=1 << 32, p=0.1, seed=1)
    assert e.value.status == 4


def test_beside_other_kernels_with_tensor_memory():
    """The whole-GPU form on one stream while the streamed row backward and the
    normalisation-GEMM, which use tensor memory too, run on two others."""
    x, g, b, dy = make(2, 30000, 256, torch.bfloat16, seed=4)
    for back in (False, True):
        assert gb.norm_group_plan(2, 30000, 256, 32, gb.BF16, back)["form"] == 2
    gen = torch.Generator(device="cuda").manual_seed(9)
    rows, drows = (torch.randn(160, 131072, device="cuda", generator=gen).bfloat16()
                   for _ in range(2))
    rg = torch.randn(131072, device="cuda", generator=gen).bfloat16()
    _, rr, _ = gb.norm_fwd(rows, rg, None, 1e-5, gb.RMS)
    a = torch.randn(4096, 1024, device="cuda", generator=gen).bfloat16()
    ag = torch.randn(1024, device="cuda", generator=gen).bfloat16()
    w = torch.randn(1024, 1024, device="cuda", generator=gen).bfloat16()
    wg, u, v = gb.norm_gemm_prepare(w, ag, None, gb.RMS)

    def group():
        y, rstd, mean = gb.norm_group_fwd(x, g, b, 32, 1e-5, "silu")
        return (y, *gb.norm_group_bwd(dy, x, g, b, rstd, mean, 32, "silu"))

    def wide():
        return gb.norm_bwd(drows, rows, rg, rr, None, gb.RMS)[:2]

    def gemm():
        return gb.norm_gemm_fwd(a, wg, u, v, 1e-5, gb.RMS)[:1]

    jobs = (group, wide, gemm)
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for s, j in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(j())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for p, q in zip(outs, want[i % 3]):
            assert torch.equal(p, q)
    assert gb.norm_get_device_error() == 0
