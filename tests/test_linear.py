"""norm_linear_fwd / norm_linear_bwd: refusals (CPU) and results against the
float64 form (GPU)."""
import ctypes

import pytest
import torch

import linear_ref as lr
import memory_bound_normalization_rmsnorm_gb300 as gb

F = 256  # a fake, aligned address: validation fails before any use
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def test_fwd_refusals():
    f = gb.lib().norm_linear_fwd
    ok = dict(x=F, ldx=64, w=F, ldw=64, b=F, r=F, ldr=32, M=4, K=64, N=32, act=0, dt=0, y=F, ldy=32,
              z=F, ldz=32, ws=None, wsb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["x"], a["ldx"], a["w"], a["ldw"], a["b"], a["r"], a["ldr"], a["M"], a["K"],
                 a["N"], a["act"], a["dt"], a["y"], a["ldy"], a["z"], a["ldz"], a["ws"], a["wsb"],
                 None)

    assert call(x=None) == 1
    assert call(w=None) == 1
    assert call(y=None) == 1
    assert call(M=0) == 2
    assert call(M=(1 << 24) + 1) == 2
    assert call(K=0) == 2
    assert call(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21) == 2
    assert call(N=0) == 2
    assert call(ldx=63) == 2                   # rows overlap
    assert call(ldw=0) == 2
    assert call(ldy=31) == 2
    assert call(ldr=-32) == 2
    assert call(ldz=8) == 2
    assert call(ldx=(1 << 32) + 8) == 2
    assert call(x=F + 1) == 3
    assert call(b=F + 1) == 3
    assert call(act=3) == 9
    assert call(act=-1) == 9
    assert call(dt=2) == 9                     # fp32
    assert call(x=F + 2) == 5                  # needs a workspace for its copy
    assert call(ldw=65) == 5
    assert call(ldw=65, ws=F, wsb=100) == 5
    assert call(ldw=65, ws=F + 8, wsb=1 << 20) == 3
    n = ctypes.c_size_t(7)
    q = gb.lib().norm_linear_fwd_workspace_bytes
    assert q(F, 64, F, 64, 4, 64, 32, ctypes.byref(n)) == 0 and n.value == 0
    assert q(F, 64, F, 65, 4, 64, 32, ctypes.byref(n)) == 0 and n.value == 32 * 64 * 2
    assert q(F + 2, 64, F, 64, 4, 64, 32, ctypes.byref(n)) == 0 and n.value == 4 * 64 * 2
    assert q(F + 2, 64, F, 64, 0, 64, 32, ctypes.byref(n)) == 2
    assert q(None, 64, F, 64, 4, 64, 32, ctypes.byref(n)) == 1
    if not torch.cuda.is_available():
        assert call() == 7
        assert call(M=1, ldx=3, ldy=0, ldr=0, ldz=0) == 7  # strides of a single row are not read


def test_bwd_refusals():
    f = gb.lib().norm_linear_bwd
    ok = dict(dy=F, lddy=32, x=F, ldx=64, w=F, ldw=64, z=F, ldz=32, M=4, K=64, N=32, act=1, dt=0,
              dx=F, lddx=64, dw=F, lddw=64, db=F, ws=F, wsb=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["dy"], a["lddy"], a["x"], a["ldx"], a["w"], a["ldw"], a["z"], a["ldz"], a["M"],
                 a["K"], a["N"], a["act"], a["dt"], a["dx"], a["lddx"], a["dw"], a["lddw"], a["db"],
                 a["ws"], a["wsb"], None)

    assert call(dy=None) == 1
    assert call(x=None) == 1
    assert call(w=None) == 1
    assert call(z=None) == 1                   # an activation needs z
    assert call(N=0) == 2
    assert call(lddy=31) == 2
    assert call(lddx=63) == 2
    assert call(ldz=1) == 2
    assert call(db=F + 2) == 3
    assert call(dy=F + 1) == 3
    assert call(act=4) == 9
    assert call(dt=2) == 9
    assert call(dx=None, dw=None, db=None) == 9
    n = ctypes.c_size_t(0)
    q = gb.lib().norm_linear_bwd_workspace_bytes
    assert q(F, 32, F, 64, F, 64, None, 0, 4, 64, 32, 1, 1, 1, 1, ctypes.byref(n)) == 1
    assert q(F, 32, None, 64, F, 64, F, 32, 4, 64, 32, 1, 1, 1, 1, ctypes.byref(n)) == 1
    assert q(F, 32, F, 64, F, 64, F, 32, 4, 64, 32, 7, 1, 1, 1, ctypes.byref(n)) == 9
    if not torch.cuda.is_available():
        assert call() == 7


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        gb.norm_linear_fwd(torch.zeros(2, 8).bfloat16(), torch.zeros(4, 8).bfloat16())


# ------------------------------------------------------------------- GPU
def _make(dtype, M, K, N, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = dict(generator=g, device="cuda")
    dt = DT[dtype]
    return dict(x=torch.randn(M, K, **r).to(dt), w=(torch.randn(N, K, **r) / K ** 0.5).to(dt),
                bias=(0.3 * torch.randn(N, **r)).to(dt), r=torch.randn(M, N, **r).to(dt),
                dy=torch.randn(M, N, **r).to(dt))


def _fwd_check(c, name, bias=True, res=True, want_z=True, **kw):
    b, r = c["bias"] if bias else None, c["r"] if res else None
    y, z = gb.norm_linear_fwd(c["x"], c["w"], b, r, name, want_z=want_z, **kw)
    (wy, wz), (ey, ez) = lr.forward(c["x"], c["w"], b, r, name)
    lr.check(y, wy, ey, "y")
    assert (z is not None) == want_z
    if want_z:
        lr.check(z, wz, ez, "z")
    return y, z


def _bwd_check(c, name, got=None, **kw):
    z = lr.forward(c["x"], c["w"], c["bias"], None, name)[0][1].to(c["x"].dtype)
    if got is None:
        got = gb.norm_linear_bwd(c["dy"], c["x"], c["w"], z if name != "none" else None, name, **kw)
    want, err, sq = lr.backward(c["dy"], c["x"], c["w"], z, name)
    for g, w, e, s, n in zip(got, want, err, (*sq, None), ("dx", "dw", "dbias")):
        if g is not None:
            lr.check(g, w, e, n, s)
    return got


SHAPES = [(1, 1, 1), (1, 64, 128), (2, 8, 16), (1, 4096, 1024), (3, 520, 264), (16, 1000, 400),
          (17, 136, 72), (48, 2048, 512), (129, 256, 384), (200, 72, 130), (65, 77, 99),
          (33, 130, 7), (7, 9, 300), (500, 640, 1288), (777, 1234, 999), (2100, 200, 1544),
          (2500, 71, 1541), (1, 16384, 256), (150, 64, 131072), (192, 40, 90001),
          (90001, 24, 40), (20000, 8, 192)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_both_directions(dtype, name, shape):
    c = _make(dtype, *shape)
    _fwd_check(c, name)
    _fwd_check(c, name, bias=False, res=False, want_z=False)
    _bwd_check(c, name)
    assert gb.norm_get_device_error() == 0


FORMS = [f"pair=1,bn={b}" for b in (64, 96, 128, 160, 192, 224, 256)]
FORMS += [f"pair=0,bn={b},splits={s}" for b, s in
          ((16, 1), (16, 8), (32, 3), (48, 2), (64, 5), (64, 1), (80, 6), (112, 4), (128, 1),
           (128, 2), (128, 7), (192, 1), (256, 4))]


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", [(5, 70, 33), (300, 600, 328), (130, 64, 264), (257, 520, 513)])
def test_every_form(form, shape, monkeypatch):
    """Each kernel form at sizes that other forms are chosen for."""
    monkeypatch.setenv("GBNORM_LINEAR", form)
    c = _make("bf16", *shape)
    _fwd_check(c, "silu")
    _fwd_check(c, "none", res=False, want_z=False)
    _fwd_check(c, "gelu", bias=False, want_z=False)
    _fwd_check(c, "gelu", res=False)
    _bwd_check(c, "gelu")
    _bwd_check(c, "none")
    assert gb.norm_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 64, 128), (2200, 136, 1544), (2200, 136, 1541)])
def test_strides_in_place_and_what_lies_around(shape):
    """Rows inside larger buffers, the residual updated in place, and nothing
    written outside."""
    M, K, N = shape
    c = _make("bf16", M, K, N)
    wide = torch.zeros(M + 3, K + 24, device="cuda", dtype=torch.bfloat16)
    wide[:M, 8:8 + K] = c["x"]
    ww = torch.zeros(N, K + 5, device="cuda", dtype=torch.bfloat16)
    ww[:, 2:2 + K] = c["w"]
    buf = torch.full((M + 2, N + 17), 5.0, device="cuda", dtype=torch.bfloat16)
    want, _ = _fwd_check(c, "gelu", want_z=False)
    c["x"], c["w"] = wide[:M, 8:8 + K], ww[:, 2:2 + K]
    for off in (0, 1, 8):
        buf.fill_(5.0)
        y = buf[1:M + 1, off:off + N]
        y.copy_(c["r"])
        got, _ = gb.norm_linear_fwd(c["x"], c["w"], c["bias"], y, "gelu", y=y)
        assert got.data_ptr() == y.data_ptr()
        assert torch.equal(y, want)
        buf[1:M + 1, off:off + N] = 5.0
        assert (buf == 5).all()
    dxb = torch.full((M, K + 3), 5.0, device="cuda", dtype=torch.bfloat16)
    dwb = torch.full((N, K + 8), 5.0, device="cuda", dtype=torch.bfloat16)
    _bwd_check(c, "silu", dx=dxb[:, 1:K + 1], dw=dwb[:, :K])
    assert (dxb[:, 0] == 5).all() and (dxb[:, K + 1:] == 5).all() and (dwb[:, K:] == 5).all()


@pytest.mark.gpu
def test_wanted_gradients_alone():
    c = _make("fp16", 70, 96, 136)
    z = lr.forward(c["x"], c["w"], c["bias"], None, "gelu")[0][1].half()
    full = gb.norm_linear_bwd(c["dy"], c["x"], c["w"], z, "gelu")
    for i, kw in enumerate((dict(want_dw=False, want_dbias=False),
                            dict(want_dx=False, want_dbias=False),
                            dict(want_dx=False, want_dw=False))):
        args = [c["x"], c["w"]]
        if i != 1:
            args[0] = None
        if i != 0:
            args[1] = None
        got = gb.norm_linear_bwd(c["dy"], *args, z, "gelu", **kw)
        for k in range(3):
            assert torch.equal(got[k], full[k]) if k == i else got[k] is None


@pytest.mark.gpu
def test_leading_dimensions_and_workspaces():
    c = _make("bf16", 24, 77, 50)
    y, _ = gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], "silu")
    y3, z3 = gb.norm_linear_fwd(c["x"].view(2, 12, 77), c["w"], c["bias"], c["r"].view(2, 12, 50),
                                "silu", want_z=True)
    assert y3.shape == z3.shape == (2, 12, 50) and torch.equal(y3.view(24, 50), y)
    one, _ = gb.norm_linear_fwd(c["x"][3], c["w"], c["bias"], c["r"][3], "silu")
    assert one.shape == (50,) and (one.float() - y[3].float()).abs().max() < 0.05
    n = gb.norm_linear_fwd_workspace_bytes(c["x"], c["w"])
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], "silu",
                                          workspace=ws)[0], y)
    with pytest.raises(gb.NormError):
        gb.norm_linear_fwd(c["x"], c["w"], c["bias"], workspace=ws[:n - 256])
    n = gb.norm_linear_bwd_workspace_bytes(c["dy"], c["x"], c["w"])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for a, b in zip(gb.norm_linear_bwd(c["dy"], c["x"], c["w"], workspace=ws),
                    gb.norm_linear_bwd(c["dy"], c["x"], c["w"])):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("pair", [0, 1])
def test_infinities_and_nans_stay_in_their_rows(pair, monkeypatch):
    monkeypatch.setenv("GBNORM_LINEAR", f"pair={pair}")
    c = _make("bf16", 150, 100, 140)
    c["x"][40, 99] = float("nan")
    c["x"][41, 0] = float("inf")
    y, _ = gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"])
    bad = ~torch.isfinite(y.float())
    assert bad[40].all() and bad[41].all() and int(bad.sum()) == 280
    # the rows behind the last and the columns behind the last hold anything
    big = torch.full((152, 104), float("nan"), device="cuda", dtype=torch.bfloat16)
    big[:150, :100] = _make("bf16", 150, 100, 140)["x"]
    c["x"] = big[:150, :100]
    _fwd_check(c, "gelu")
    _bwd_check(c, "none")


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activations_at_extreme_arguments(name):
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5, -5, 9, -9, 13, -13, 40, -40, 87, -87, 90, -90,
                      300, -300, 3e4, -3e4, 1e19, -1e19, 3e38, -3e38], device="cuda")
    x, w = v.bfloat16()[:, None].contiguous(), torch.ones(1, 1, device="cuda").bfloat16()
    y, z = gb.norm_linear_fwd(x, w, None, None, name, want_z=True)
    assert torch.equal(z, x)
    want = lr.act(x.double(), name)
    assert torch.isfinite(y.float()).all()
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all()
    dx, _, db = gb.norm_linear_bwd(torch.ones_like(y), x, w, z, name)
    slope, mag = lr.act_grad(x.double().clamp(-1e3, 1e3), name)
    assert ((dx.double() - slope).abs() <= 2.0 ** -8 * slope.abs() + 2.0 ** -18 * mag + 1e-30).all()


@pytest.mark.gpu
def test_binding_refusals():
    c = _make("bf16", 6, 16, 24)
    fwd, bwd = gb.norm_linear_fwd, gb.norm_linear_bwd
    for args, word in (((c["x"].float(), c["w"]), "bfloat16 or float16"),
                       ((c["x"], c["w"].half()), "w must be"),
                       ((c["x"], c["w"].t()), "w has shape"),
                       ((c["x"], c["w"].t().contiguous().t()), "contiguous"),
                       ((c["x"][:, ::2], c["w"][:, ::2]), "contiguous"),
                       ((c["x"], c["w"], c["bias"][:5]), "bias has shape"),
                       ((c["x"], c["w"], None, c["r"][:2]), "r has shape"),
                       ((c["x"], c["w"], None, None, "tanh"), "act must be"),
                       ((c["x"], c["w"].cpu()), "CUDA")):
        with pytest.raises(ValueError, match=word):
            fwd(*args)
    for args, word in (((c["dy"], None, c["w"]), "x must be given"),
                       ((c["dy"], c["x"], None), "w must be given"),
                       ((c["dy"], c["x"][:3], c["w"]), "x has shape"),
                       ((c["dy"][:, :7], c["x"], c["w"]), "w has shape")):
        with pytest.raises(ValueError, match=word):
            bwd(*args)
    with pytest.raises(gb.NormError) as e:
        bwd(c["dy"], c["x"], c["w"], None, "gelu")
    assert e.value.status == 1
    with pytest.raises(gb.NormError) as e:
        bwd(c["dy"], c["x"], c["w"], want_dx=False, want_dw=False, want_dbias=False)
    assert e.value.status == 9
    with pytest.raises(gb.NormError):
        fwd(c["x"][:0], c["w"])


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    sizes = [(3, 512, 256), (300, 256, 520), (2100, 328, 1544)]
    cases = [_make("bf16", *s) for s in sizes]
    zs = [c["r"].clone() for c in cases]

    def run(stream=None):
        out = []
        for c, z in zip(cases, zs):
            out += gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], "gelu", want_z=True,
                                      stream=stream)
            out += gb.norm_linear_bwd(c["dy"], c["x"], c["w"], z, "gelu", stream=stream)
        return out

    first = [t.clone() for t in run()]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # two streams at once
        a = run()
    b = run(stream=other)
    torch.cuda.synchronize()
    for x, y, w in zip(a, b, first):
        assert torch.equal(x, w) and torch.equal(y, w)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = run()
        graphs.append((gr, outs))
    for c, z in zip(cases, zs):
        c["x"].mul_(0.5)
        z.mul_(2)
    for gr, _ in graphs:
        gr.replay()
    want = run()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for x, w in zip(outs, want):
            assert torch.equal(x, w)
    assert not torch.equal(want[0], first[0])
    assert gb.norm_get_device_error() == 0


@pytest.mark.gpu
def test_first_call_of_a_size_inside_a_capture():
    c = _make("fp16", 37, 192, 336)
    z = c["r"]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.empty(1, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        y, _ = gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], "silu")
        got = gb.norm_linear_bwd(c["dy"], c["x"], c["w"], z, "silu")
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], "silu")[0])
    for a, b in zip(got, gb.norm_linear_bwd(c["dy"], c["x"], c["w"], z, "silu")):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_many_threads_and_sizes():
    """Calls of new sizes from several threads at once, each on its stream."""
    import threading

    sizes = [(5 + 7 * i, 40 + 8 * i, 24 + 16 * i) for i in range(12)]
    cases = [_make("bf16", *s, seed=i) for i, s in enumerate(sizes)]
    outs = {}

    def work(t):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for i in range(t, 12, 4):
                outs[i] = gb.norm_linear_fwd(cases[i]["x"], cases[i]["w"], cases[i]["bias"])[0]
        s.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, c in enumerate(cases):
        (wy, _), (ey, _) = lr.forward(c["x"], c["w"], c["bias"], None, "none")
        lr.check(outs[i], wy, ey, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2304, 4096, 512), (512, 256, 4096), (40, 2048, 512),
                                   (300, 640, 4099)])
def test_backward_between_writers_and_readers(shape):
    """Every gradient is read by the kernel behind, and the operands are written by
    the one before, over and over in the same buffers."""
    M, K, N = shape
    c = _make("bf16", M, K, N)
    dx, dw = torch.empty_like(c["x"]), torch.empty_like(c["w"])
    db = torch.empty(N, device="cuda")
    keep = dict(p=0.0, seed=1)
    want = {}
    for i in range(12):
        f = 1.0 + i % 3  # exact factors: the gradients scale with dy, and dw with x
        dy, x = c["dy"] * f, gb.norm_dropout(c["x"] * f, **keep)
        gb.norm_linear_bwd(dy, x, c["w"], dx=dx, dw=dw, dbias=db)
        got = (gb.norm_dropout(dx, **keep), gb.norm_dropout(dw, **keep), gb.norm_dropout(db, **keep))
        for t in (dx, dw, db):
            t.fill_(float("nan"))
        if i < 3:
            want[f] = [g.clone() for g in got]
        else:
            for g, w in zip(got, want[f]):
                assert torch.equal(g, w)
    torch.cuda.synchronize()
    full = gb.norm_linear_bwd(c["dy"], c["x"], c["w"])
    for g, w in zip(want[1.0], full):
        assert torch.equal(g, w)


@pytest.mark.gpu
def test_beside_other_kernels_that_hold_tensor_memory():
    """Split-form clusters on one stream, pair-form and the normalisation-GEMM on
    others, many at once."""
    c = _make("bf16", 40, 2048, 2048)
    big = _make("bf16", 2304, 512, 2048)
    gamma = torch.ones(512, device="cuda").bfloat16()
    wg, u, v = gb.norm_gemm_prepare(big["w"][:, :512].contiguous(), gamma)
    want = [gb.norm_linear_fwd(c["x"], c["w"])[0], gb.norm_linear_fwd(big["x"], big["w"])[0],
            gb.norm_gemm_fwd(big["x"], wg)[0]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append((i, [lambda: gb.norm_linear_fwd(c["x"], c["w"])[0],
                                 lambda: gb.norm_linear_fwd(big["x"], big["w"])[0],
                                 lambda: gb.norm_gemm_fwd(big["x"], wg)[0]][i]()))
    torch.cuda.synchronize()
    for i, o in outs:
        assert torch.equal(o, want[i])
    assert gb.norm_get_device_error() == 0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Rows so far apart that the last lie beyond 2^31 elements."""
    M, K, N, step = 3, 64, 136, 1 << 30
    c = _make("bf16", M, K, N)
    flat = torch.zeros((M - 1) * step + 256, device="cuda", dtype=torch.bfloat16)
    x = flat.as_strided((M, K), (step, 1))
    x.copy_(c["x"])
    c["x"] = x
    out = flat.as_strided((M, N), (step, 1), 64)
    y, _ = gb.norm_linear_fwd(c["x"], c["w"], c["bias"], c["r"], y=out)
    (wy, _), (ey, _) = lr.forward(c["x"], c["w"], c["bias"], c["r"], "none")
    lr.check(y, wy, ey, "y")
