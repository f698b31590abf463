"""norm_rope_fwd / norm_rope_bwd: refusals (CPU) and results against the float64
form (GPU)."""
import ctypes

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb
import rope_ref as rr

F = 16  # a fake, aligned address: validation fails before any use
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _heads(data=F, ts=64, hs=16):
    return gb._binding.Heads(data, ts, hs)


def _ref(h):
    return None if h is None else ctypes.byref(h)


def test_fwd_refusals():
    f = gb.lib().norm_rope_fwd
    ok = dict(q=_heads(), k=_heads(), T=3, Hq=4, Hk=4, D=16, rd=16, pos=F, bits=64, ps=3, f=F,
              ax=bytes(8), axes=1, inter=0, gq=F, gk=F, bq=None, bk=None, eps=1e-6, mode=0, dt=0,
              yq=_heads(), yk=_heads())

    def call(**kw):
        a = dict(ok, **kw)
        return f(_ref(a["q"]), _ref(a["k"]), a["T"], a["Hq"], a["Hk"], a["D"], a["rd"], a["pos"],
                 a["bits"], a["ps"], a["f"], a["ax"], a["axes"], a["inter"], a["gq"], a["gk"],
                 a["bq"], a["bk"], a["eps"], a["mode"], a["dt"], _ref(a["yq"]), _ref(a["yk"]), None)

    assert call(q=None) == 1
    assert call(k=None) == 1
    assert call(yk=_heads(None)) == 1
    assert call(pos=None) == 1
    assert call(f=None) == 1
    assert call(gk=None) == 1                  # one side normalised only
    assert call(gq=None) == 1
    assert call(axes=2, ax=None) == 1
    assert call(T=0) == 2
    assert call(T=(1 << 31) + 1) == 2
    assert call(Hq=0) == 2
    assert call(Hk=-1) == 2
    assert call(D=258, rd=16) == 2
    assert call(D=1) == 2
    assert call(rd=15) == 2
    assert call(rd=18) == 2                    # more turned elements than the head has
    assert call(rd=0) == 2
    assert call(q=_heads(ts=-64)) == 2
    assert call(yq=_heads(ts=63)) == 2         # output tokens overlap
    assert call(yq=_heads(hs=15)) == 2         # output heads overlap
    assert call(yq=_heads(ts=0)) == 2
    assert call(yq=_heads(F + 1)) == 3
    assert call(pos=F + 4) == 3
    assert call(pos=F + 2, bits=32) == 3
    assert call(f=F + 4) == 3
    assert call(gq=F + 1) == 3
    assert call(mode=2) == 4
    assert call(bq=F) == 4                     # beta with RMSNorm
    assert call(mode=1, gq=None, gk=None, bq=F) == 4
    assert call(axes=0) == 9
    assert call(axes=5) == 9
    assert call(axes=2, ax=bytes([0, 1, 2, 0, 0, 0, 0, 0])) == 9   # an axis that is not there
    assert call(bits=16) == 9
    assert call(inter=2) == 9
    assert call(eps=-1.0) == 9
    assert call(eps=float("nan")) == 9
    assert call(dt=3) == 9
    assert call(ps=-1) == 9
    assert call(Hk=0, k=None, yk=None) == 9    # gamma_k without keys
    if not torch.cuda.is_available():
        assert call() == 7
        assert call(Hk=0, k=None, yk=None, gk=None) == 7
        assert call(q=_heads(F + 2), yq=_heads(ts=67, hs=16)) == 7  # any element alignment


def test_bwd_refusals():
    f = gb.lib().norm_rope_bwd
    h = _heads()
    ok = dict(dyq=h, dyk=h, q=h, k=h, T=3, Hq=4, Hk=4, D=16, rd=16, pos=F, bits=64, ps=3, f=F,
              ax=bytes(8), axes=1, inter=0, gq=F, gk=F, eps=1e-6, mode=0, dt=0, dq=h, dk=h, dgq=F,
              dgk=F, dbq=None, dbk=None, ws=F, wsb=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return f(_ref(a["dyq"]), _ref(a["dyk"]), _ref(a["q"]), _ref(a["k"]), a["T"], a["Hq"],
                 a["Hk"], a["D"], a["rd"], a["pos"], a["bits"], a["ps"], a["f"], a["ax"], a["axes"],
                 a["inter"], a["gq"], a["gk"], a["eps"], a["mode"], a["dt"], _ref(a["dq"]),
                 _ref(a["dk"]), a["dgq"], a["dgk"], a["dbq"], a["dbk"], a["ws"], a["wsb"], None)

    assert call(dyq=None) == 1
    assert call(dk=None) == 1
    assert call(q=None) == 1                   # the statistics need the inputs
    assert call(dgk=None) == 1
    assert call(gk=None) == 1
    assert call(T=0) == 2
    assert call(dq=_heads(ts=0)) == 2
    assert call(dgq=F + 2) == 3
    assert call(mode=7) == 4
    assert call(dbq=F) == 4                    # dbeta with RMSNorm
    assert call(gq=None, gk=None) == 4         # dgamma without normalisation
    assert call(dt=9) == 9
    assert call(Hk=0) == 9                     # gamma_k without keys
    n = ctypes.c_size_t(7)
    w = gb.lib().norm_rope_bwd_workspace_bytes
    assert w(3, 4, 4, 16, 0, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert w(3, 4, 4, 300, 1, 0, ctypes.byref(n)) == 2
    assert w(3, 4, 4, 16, 1, 0, None) == 1
    if not torch.cuda.is_available():
        assert call() == 7
        assert call(gq=None, gk=None, dgq=None, dgk=None, q=None, k=None, ws=None, wsb=0) == 7


def test_binding_refuses_host_tensors():
    q = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gb.norm_rope_fwd(q, None, torch.zeros(2, dtype=torch.int64), torch.ones(4).double())


# ------------------------------------------------------------------- GPU
def _make(dtype, mode, T, Hq, Hk, D, rd, axes=1, inter=False, packed=False, pos32=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = dict(generator=g, device="cuda")
    dt = DT[dtype]
    if packed:
        rows = torch.randn(T, (Hq + 2 * Hk) * D, **r).to(dt)
        q, k = rows[:, :Hq * D].view(T, Hq, D), rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    else:
        q, k = torch.randn(T, Hq, D, **r).to(dt), torch.randn(T, Hk, D, **r).to(dt)
    par = {}
    for n in ("q", "k"):
        has = n == "q" or Hk > 0
        norm, layer = has and mode != "none", has and mode == "layer"
        par["gamma_" + n] = (1 + 0.2 * torch.randn(D, **r)).to(dt) if norm else None
        par["beta_" + n] = (0.2 * torch.randn(D, **r)).to(dt) if layer else None
    sec = rr.sections(rd // 2, axes)
    pos = torch.randint(0, 1 << 18, (T,) if axes == 1 else (axes, T), **r)
    if pos32:
        pos = pos.int()
    inv = torch.tensor([10000.0 ** (-2 * i / rd) for i in range(rd // 2)], dtype=torch.float64,
                       device="cuda")
    return dict(q=q, k=k if Hk else None, pos=pos, inv=inv, par=par, sec=sec, inter=inter,
                layer=mode == "layer", mode=gb.LAYER if mode == "layer" else gb.RMS,
                ang=rr.angles(pos, inv, sec))


def _fwd(c, eps=1e-6, **kw):
    return gb.norm_rope_fwd(c["q"], c["k"], c["pos"], c["inv"], **c["par"], eps=eps, mode=c["mode"],
                            sections=c["sec"], interleaved=c["inter"], **kw)


def _bwd(c, dyq, dyk, eps=1e-6, **kw):
    return gb.norm_rope_bwd(dyq, dyk, c["q"], c["k"], c["pos"], c["inv"], c["par"]["gamma_q"],
                            c["par"]["gamma_k"], eps, c["mode"], sections=c["sec"],
                            interleaved=c["inter"], **kw)


def _check_fwd(c, yq, yk, eps=1e-6):
    for n, y in (("q", yq), ("k", yk)):
        if c[n] is None:
            assert y is None
            continue
        want, mag = rr.forward(c[n], c["ang"], c["inter"], c["par"]["gamma_" + n],
                               c["par"]["beta_" + n], eps, c["layer"])
        rr.check(y, want, mag, rr.ARITH_Y, "y" + n)


def _check_bwd(c, dys, got, eps=1e-6):
    dq, dk, dgq, dgk, dbq, dbk = got
    for n, dy, dx, dg, db in (("q", dys[0], dq, dgq, dbq), ("k", dys[1], dk, dgk, dbk)):
        if c[n] is None:
            assert dx is None and dg is None and db is None
            continue
        gamma = c["par"]["gamma_" + n]
        want, mag = rr.backward(dy, c[n], c["ang"], c["inter"], gamma, eps, c["layer"])
        rr.check(dx, want[0], mag[0], rr.ARITH_G, "d" + n)
        assert (dg is None) == (gamma is None)
        assert (db is None) == (not c["layer"])
        if dg is not None:
            rr.check(dg, want[1], mag[1], rr.ARITH_G, "dgamma_" + n)
        if db is not None:
            rr.check(db, want[2], mag[2], rr.ARITH_G, "dbeta_" + n)


SHAPES = [
    # T, Hq, Hk, D, rd, axes, inter, packed, pos32
    (1, 1, 0, 2, 2, 1, False, False, False),        # the smallest call
    (1, 32, 8, 128, 128, 3, False, True, False),    # one token
    (3, 5, 1, 64, 64, 2, True, False, True),
    (7, 3, 3, 72, 36, 1, False, False, False),      # 18 pairs: four-byte chunks
    (7, 3, 2, 72, 72, 2, True, True, True),
    (5, 2, 2, 10, 6, 3, False, False, False),       # 3 pairs, 4 unturned: single elements
    (6, 4, 1, 11, 10, 1, True, False, False),       # odd head
    (19, 4, 2, 256, 256, 4, False, True, False),
    (19, 4, 2, 256, 128, 4, True, False, False),
    (13, 2, 1, 254, 254, 1, False, False, False),   # 127 pairs
    (13, 2, 1, 254, 130, 2, True, False, False),
    (33, 16, 16, 80, 80, 2, True, False, False),
    (1000, 6, 2, 96, 96, 3, False, True, True),     # more warps than one wave of CTAs
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", ["none", "rms", "layer"])
@pytest.mark.parametrize("shape", SHAPES)
def test_both_directions(dtype, mode, shape):
    T, Hq, Hk, D, rd, axes, inter, packed, pos32 = shape
    c = _make(dtype, mode, T, Hq, Hk, D, rd, axes, inter, packed and Hk > 0, pos32)
    yq, yk = _fwd(c)
    _check_fwd(c, yq, yk)
    g = torch.Generator(device="cuda").manual_seed(5)
    dys = [None if t is None else torch.randn(t.shape, generator=g, device="cuda").to(t.dtype)
           for t in (c["q"], c["k"])]
    _check_bwd(c, dys, _bwd(c, *dys))


# Heads of one to thirty-two lanes with one to three units each, turned whole and
# in part, in both pair layouts.
LANES = [
    (9, 2, 1, 8, 8, 1), (9, 3, 2, 16, 16, 1), (9, 3, 1, 16, 8, 1), (9, 2, 2, 24, 16, 1),
    (21, 3, 2, 32, 32, 2), (70, 3, 2, 48, 48, 3), (21, 3, 2, 48, 32, 1), (21, 2, 1, 80, 48, 1),
    (11, 5, 3, 96, 32, 1), (21, 3, 2, 96, 96, 2), (23, 2, 2, 104, 96, 2), (13, 2, 1, 112, 112, 1),
    (23, 2, 2, 144, 144, 3), (11, 3, 1, 160, 160, 3), (11, 3, 1, 192, 192, 1), (11, 2, 1, 192, 64, 1),
    (11, 2, 1, 208, 176, 2), (5, 2, 1, 256, 256, 1), (12000, 2, 1, 80, 80, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("mode", ["none", "rms", "layer"])
@pytest.mark.parametrize("shape", LANES)
def test_lanes_and_units(shape, mode, inter):
    T, Hq, Hk, D, rd, axes = shape
    for dtype in ("bf16", "fp32"):
        c = _make(dtype, mode, T, Hq, Hk, D, rd, axes, inter, True)
        _check_fwd(c, *_fwd(c))
        dys = [torch.randn_like(c["q"]), torch.randn_like(c["k"])]
        _check_bwd(c, dys, _bwd(c, *dys))


@pytest.mark.gpu
@pytest.mark.parametrize("pos", [2 ** 31 - 1, -1, -2 ** 31, 2 ** 20 + 12345])
def test_far_positions(pos):
    c = _make("fp32", "none", 4, 2, 1, 128, 128)
    for bits in (torch.int64, torch.int32):
        c["pos"] = torch.tensor([pos, 0, 1, pos], device="cuda").to(bits)
        # inv_freq of a few bits: pos * inv_freq is exact in float64
        c["inv"] = torch.tensor([2.0 ** -(i % 16) * (1 + (i % 3) / 4) for i in range(64)],
                                device="cuda", dtype=torch.float64)
        c["ang"] = rr.angles(c["pos"], c["inv"], None)
        _check_fwd(c, *_fwd(c))


@pytest.mark.gpu
def test_in_place_and_strided_outputs():
    for dtype in ("bf16", "fp32"):
        c = _make(dtype, "rms", 37, 4, 2, 64, 64, packed=True)
        want = [t.clone() for t in _fwd(c)]
        # a larger buffer: what lies between and behind the rows stays
        buf = torch.full((40, 9, 64), 7.0, device="cuda", dtype=DT[dtype])
        yq, yk = buf[:37, 1:5], buf[:37, 6:8]
        got = _fwd(c, yq=yq, yk=yk)
        assert got[0].data_ptr() == yq.data_ptr()
        assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
        rest = torch.ones(40, 9, dtype=torch.bool, device="cuda")
        rest[:37, 1:5] = rest[:37, 6:8] = False
        assert (buf[rest] == 7).all()
        _fwd(c, yq=c["q"], yk=c["k"])
        assert torch.equal(c["q"], want[0]) and torch.equal(c["k"], want[1])


@pytest.mark.gpu
def test_gradient_in_place_of_the_incoming_one():
    c = _make("bf16", "layer", 21, 4, 2, 64, 32)
    dys = [torch.randn_like(c["q"]), torch.randn_like(c["k"])]
    want = _bwd(c, *dys)
    a, b = dys[0].clone(), dys[1].clone()
    got = _bwd(c, a, b, dq=a, dk=b)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_addresses_and_strides_of_any_element(offset):
    c = _make("bf16", "rms", 9, 3, 2, 64, 64)
    flat = torch.zeros(9 * (5 * 64 + 3) + 8, device="cuda", dtype=torch.bfloat16)
    rows = flat[offset:offset + 9 * (5 * 64 + 3)].view(9, 5 * 64 + 3)
    rows[:, :192] = c["q"].reshape(9, -1)
    rows[:, 192:320] = c["k"].reshape(9, -1)
    want = _fwd(c)
    c["q"], c["k"] = rows[:, :192].view(9, 3, 64), rows[:, 192:320].view(9, 2, 64)
    _check_fwd(c, *_fwd(c))
    assert (_fwd(c)[0].float() - want[0].float()).abs().max() < 0.05


@pytest.mark.gpu
def test_infinities_and_nans_stay_in_their_rows():
    c = _make("fp32", "none", 4, 2, 1, 16, 8)
    c["q"][1, 0, 12] = float("inf")            # an element that does not turn
    c["q"][2, 1, 13] = float("nan")
    yq, yk = _fwd(c)
    assert torch.isinf(yq[1, 0, 12]) and torch.isnan(yq[2, 1, 13])
    bad = ~torch.isfinite(yq)
    assert int(bad.sum()) == 2 and torch.isfinite(yk).all()
    c = _make("bf16", "rms", 4, 3, 1, 64, 64)
    c["q"][1, 2, 3] = float("nan")
    yq, yk = _fwd(c)
    bad = ~torch.isfinite(yq)
    assert bad[1, 2].all() and int(bad.sum()) == 64 and torch.isfinite(yk).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["rms", "layer"])
def test_zero_and_constant_rows(mode):
    c = _make("bf16", mode, 5, 3, 3, 64, 64)
    c["q"][2] = 0
    c["k"][3] = 1.5
    _check_fwd(c, *_fwd(c))
    dys = [torch.randn_like(c["q"]), torch.randn_like(c["k"])]
    _check_bwd(c, dys, _bwd(c, *dys))
    # eps = 0 and rows that fill only part of the warps: the lanes beyond the
    # last head add nothing
    c = _make("fp32", mode, 5, 3, 3, 64, 64)
    dys = [torch.randn_like(c["q"]), torch.randn_like(c["k"])]
    _check_fwd(c, *_fwd(c, eps=0.0), eps=0.0)
    _check_bwd(c, dys, _bwd(c, *dys, eps=0.0), eps=0.0)


@pytest.mark.gpu
def test_leading_dimensions_and_given_outputs():
    c = _make("fp16", "layer", 24, 4, 2, 32, 32, axes=3)
    flat = _fwd(c)
    dys = [torch.randn_like(c["q"]), torch.randn_like(c["k"])]
    flat_b = _bwd(c, *dys)
    d = dict(c, q=c["q"].view(2, 12, 4, 32), k=c["k"].view(2, 12, 2, 32),
             pos=c["pos"].view(3, 2, 12))
    got = _fwd(d)
    assert got[0].shape == (2, 12, 4, 32)
    assert torch.equal(got[0].view_as(flat[0]), flat[0])
    dg = torch.empty(32, device="cuda")
    back = _bwd(d, dys[0].view_as(d["q"]), dys[1].view_as(d["k"]), dgamma_k=dg, want_dbeta=False)
    assert back[3].data_ptr() == dg.data_ptr() and back[4] is None and back[5] is None
    assert torch.equal(dg, flat_b[3]) and torch.equal(back[0].view_as(flat_b[0]), flat_b[0])
    n = gb.norm_rope_bwd_workspace_bytes(24, 4, 2, 32, True, gb.LAYER)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for x, y in zip(_bwd(c, *dys, workspace=ws), flat_b):
        assert torch.equal(x, y)
    with pytest.raises(gb.NormError):
        _bwd(c, *dys, workspace=ws[:n - 16])


@pytest.mark.gpu
def test_binding_refusals():
    c = _make("bf16", "rms", 4, 2, 1, 16, 16, axes=2)
    call = lambda **kw: _fwd(dict(c, **kw))  # noqa: E731
    for kw, word in ((dict(q=c["q"].transpose(1, 2)), "contiguous"),
                     (dict(k=c["k"][:3]), "k has shape"),
                     (dict(k=c["k"].half()), "k must be"),
                     (dict(inv=c["inv"].float()), "inv_freq"),
                     (dict(sec=(4, 5)), "sections"),
                     (dict(sec=(4, 3)), "sections"),
                     (dict(sec=(4, -1, 5)), "sections"),
                     (dict(sec=(1, 1, 1, 1, 4)), "sections"),
                     (dict(pos=c["pos"][:1]), "pos has shape"),
                     (dict(pos=c["pos"].float()), "int32 or int64"),
                     (dict(pos=c["pos"].cpu()), "pos must be on"),
                     (dict(pos=c["pos"].t().contiguous().t()), "contiguous")):
        with pytest.raises(ValueError, match=word):
            call(**kw)
    with pytest.raises(gb.NormError) as e:     # no tokens
        call(q=c["q"][:0], k=c["k"][:0], pos=c["pos"][:, :0])
    assert e.value.status in (1, 2)
    with pytest.raises(gb.NormError) as e:     # beta with RMSNorm
        _fwd(dict(c, par=dict(c["par"], beta_q=c["par"]["gamma_q"])))
    assert e.value.status == 4
    with pytest.raises(ValueError, match="yq has shape"):
        _fwd(c, yq=c["q"][:3])


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    c = _make("bf16", "layer", 300, 8, 2, 128, 128, axes=3, packed=True)
    dys = [torch.randn(c[n].shape, device="cuda").bfloat16() for n in ("q", "k")]
    first = [t.clone() for t in (*_fwd(c), *_bwd(c, *dys))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [*_fwd(c), *_bwd(c, *dys)]
    handed = [*_fwd(c, stream=side), *_bwd(c, *dys, stream=side)]
    side.synchronize()
    for a, b, w in zip(again, handed, first):
        assert torch.equal(a, w) and torch.equal(b, w)
    # two captured graphs replayed in turn; the inputs change between replays
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = [*_fwd(c), *_bwd(c, *dys)]
        graphs.append((gr, outs))
    c["pos"] += 17
    c["q"].mul_(0.5)
    c["ang"] = rr.angles(c["pos"], c["inv"], c["sec"])
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        _check_fwd(c, *outs[:2])
        _check_bwd(c, dys, outs[2:])


@pytest.mark.gpu
def test_rows_beyond_32_bit_offsets():
    """A row stride that puts the last tokens beyond 2^31 elements."""
    T, step = 3, 1 << 30
    flat = torch.zeros((T - 1) * step + 256, device="cuda", dtype=torch.bfloat16)
    c = _make("bf16", "rms", T, 2, 1, 128, 128)
    q = flat.as_strided((T, 2, 128), (step, 128, 1))
    q.copy_(c["q"])
    c["q"] = q
    _check_fwd(c, *_fwd(c))
