"""norm_dropout and norm_dropout_add_fwd / _bwd against the mask reference
(bit for bit), the fp64 oracle (the parity tolerances) and each other."""
import numpy as np
import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb
from memory_bound_normalization_rmsnorm_gb300 import workloads as wl

import dropout_ref as dref
import oracle
import parity_util as pu
import tolerances

pytestmark = pytest.mark.gpu

SEED, OFF = 0x9E3779B97F4A7C15, (5 << 32) + 11
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _x(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 15, 16, 4096, 8191, 8192, 8195, 100003])
def test_dropout_bitwise(dtype, n):
    x = _x((n,), dtype, n)
    for p in (0.0, 0.1, 0.5, 0.9):
        got = gb.norm_dropout(x.cuda(), p, SEED, OFF)
        want = dref.drop_f32(x, p, SEED, OFF).to(dtype)
        assert got.dtype == dtype and torch.equal(got.cpu(), want), (n, p)
    assert torch.equal(gb.norm_dropout(x.cuda(), 0.0, SEED).cpu(), x)


def test_dropout_backward_is_the_same_call():
    """y = m * x with the mask m: the gradient of sum(y * dy) is m * dy."""
    x, dy = _x((37, 53), torch.float32, 1).cuda(), _x((37, 53), torch.float32, 2).cuda()
    y = gb.norm_dropout(x, 0.3, SEED, OFF)
    dx = gb.norm_dropout(dy, 0.3, SEED, OFF)
    k = dref.keep(x.shape, 0.3, SEED, OFF).cuda()
    assert torch.equal(y != 0, k & (x != 0)) and torch.equal(dx != 0, k & (dy != 0))
    assert torch.equal(dx, torch.where(k, dy * float(dref.scale(0.3)), 0.0))


def test_dropout_of_infinities_and_nan():
    """Dropped elements are +0 whatever they held; kept ones keep it."""
    p = 0.5
    for v in (float("nan"), float("inf"), -float("inf"), -1.0):
        x = torch.full((1000,), v, dtype=torch.bfloat16)
        y = gb.norm_dropout(x.cuda(), p, 3, 4).cpu().float()
        k = dref.keep(x.shape, p, 3, 4)
        z = y[~k]
        assert torch.equal(z, torch.zeros_like(z)) and not torch.signbit(z).any()
        assert torch.isnan(y[k]).all() if v != v else (y[k] == 2 * v).all()


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
def test_dropout_in_place_and_stays_in_bounds(dtype):
    n, pad = 5003, 64
    x = _x((n,), dtype, 3)
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    view = buf[pad:pad + n]
    view.copy_(x)
    out = gb.norm_dropout(view, 0.25, SEED, OFF, y=view)
    assert out.data_ptr() == view.data_ptr()
    assert torch.equal(view.cpu(), dref.drop_f32(x, 0.25, SEED, OFF).to(dtype))
    assert (buf[:pad] == 7).all() and (buf[pad + n:] == 7).all()


def test_dropout_beyond_32_bit_elements():
    """Element indices past 2^32: block counters keep their high word in
    place and addresses do not wrap."""
    n = (1 << 32) + 8 * 4 + 5
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = gb.norm_dropout(x, 0.1, SEED, OFF, y=x)
    for first in (0, (1 << 31) - 64, (1 << 32) - 64, n - n % 8 - 32):
        m = min(100, n - first)
        want = dref.drop_f32(torch.ones(m, dtype=torch.bfloat16), 0.1, SEED, OFF, first=first)
        assert torch.equal(y[first:first + m].cpu(), want.to(torch.bfloat16)), first
    del x, y
    torch.cuda.empty_cache()


def test_offset_word_on_the_device_and_graph_replay():
    """The device word is added to offset when the kernel runs: a replayed
    graph draws the mask of the word's present value."""
    x = _x((4096,), torch.bfloat16, 5)
    xg, y = x.cuda(), torch.empty(4096, dtype=torch.bfloat16, device="cuda")
    word = torch.zeros(1, dtype=torch.int64, device="cuda")
    gb.norm_dropout(xg, 0.2, SEED, OFF, offset_dev=word, y=y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gb.norm_dropout(xg, 0.2, SEED, OFF, offset_dev=word, y=y)
    for v in (0, 1, 1 << 33):
        word.fill_(v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), dref.drop_f32(x, 0.2, SEED, OFF + v).to(torch.bfloat16))


# ------------------------------------------------- dropout + residual add
def _add_case(mode, M, N, seed):
    base = wl.WORKLOADS["layer_32768x4096" if mode else "rms_262144x1024_outliers"]
    case = wl.like(base, M, N)
    return case, wl.make_residual_inputs(case, "cpu", seed=seed)


def _run_add(ins, case, mode, p, **kw):
    x, r, g, b, dy, dh = [None if t is None else t.cuda() for t in ins]
    rng = dict(p=p, seed=SEED, offset=OFF, **kw)
    h, y, rstd, mean = gb.norm_dropout_add_fwd(x, r, g, b, case.eps, mode, **rng)
    dx, dr, dg, db = gb.norm_dropout_add_bwd(dy, dh, h, g, rstd, mean, mode, **rng)
    torch.cuda.synchronize()
    return h, y, rstd, mean, dx, dr, dg, db


def _check_add(ins, case, mode, p, outs, label, rows=None):
    x, r, g, b, dy, dh = ins
    h, y, rstd, mean, dx, dr, dg, db = outs
    eps64 = float(np.float32(case.eps))
    # h: one float32 product, one float32 sum, one rounding -- bit for bit
    href = (dref.drop_f32(x, p, SEED, OFF) + r.float()).to(torch.bfloat16)
    assert torch.equal(h.cpu(), href), f"{label}: h"
    hb, gbits, dyb, dhb = (wl.bf16_bits(t) for t in (href, g, dy, dh))
    bb = None if b is None else wl.bf16_bits(b)
    y_ref, r_ref, m_ref = oracle.fwd_bf16(hb, gbits, bb, eps64, mode)
    dr_ref = oracle.add_bwd_dx_bf16(dyb, hb, dhb, gbits, eps64, mode)
    fac = dref.keep(x.shape, p, SEED, OFF).double().numpy() * (65536.0 / (65536 - dref.threshold(p)))
    dg_ref, db_ref, dg_abs, db_abs = oracle.param_grads_bf16(dyb, hb, gbits, eps64, mode)
    tolerances.check_t1(pu.f64(y), y_ref, f"{label} y")
    tolerances.check_t1(pu.f64(dr), dr_ref, f"{label} dr")
    tolerances.check_t1(pu.f64(dx), dr_ref * fac, f"{label} dx")
    assert (pu.f64(dx)[fac == 0] == 0).all()
    tolerances.check_t2(pu.f64(rstd), r_ref, None, f"{label} rstd")
    tolerances.check_t2(pu.f64(dg), dg_ref, dg_abs, f"{label} dgamma")
    if mode:
        hs = oracle.bf16_bits_to_f64(hb)
        tolerances.check_t2(pu.f64(mean), m_ref, np.abs(hs).mean(axis=1), f"{label} mean")
        tolerances.check_t2(pu.f64(db), db_ref, db_abs, f"{label} dbeta")
    else:
        assert mean is None and db is None


# register-resident rows (exact and ragged splits), long rows, clusters
ADD_SHAPES = [(1, 8), (1, 4096), (3, 24), (257, 256), (501, 776), (129, 1024), (203, 2048),
              (301, 4096), (97, 5120), (61, 8192), (35, 8200), (33, 16384), (9, 24576),
              (7, 32768), (5, 65536), (3, 131072), (2, 262144)]


@pytest.mark.parametrize("mode", [0, 1], ids=["rms", "layer"])
@pytest.mark.parametrize("M,N", ADD_SHAPES)
def test_dropout_add_parity(mode, M, N):
    case, ins = _add_case(mode, M, N, M * 7 + N)
    outs = _run_add(ins, case, mode, 0.1)
    _check_add(ins, case, mode, 0.1, outs, f"{mode}:{M}x{N}")
    assert gb.norm_get_device_error() == 0


@pytest.mark.parametrize("mode,M,N", [(1, 301, 4096), (0, 61, 776), (1, 5, 65536)])
def test_dropout_add_is_dropout_then_add(mode, M, N):
    """The same mask as norm_dropout's, y and the statistics exactly those of
    norm_fwd-on-h up to plans, and dx = dropout of the unrounded dr."""
    case, ins = _add_case(mode, M, N, 17)
    h, y, rstd, mean, dx, dr, dg, db = _run_add(ins, case, mode, 0.25)
    x, r, g, b, dy, dh = [None if t is None else t.cuda() for t in ins]
    k = gb.norm_dropout(torch.ones_like(x), 0.25, SEED, OFF) != 0
    assert torch.equal(dx != 0, k & (dr != 0))
    h2, y2, rs2, m2 = gb.norm_add_fwd(torch.where(k, x, 0), r, g, b, case.eps, mode)
    assert torch.equal(h[~k], h2[~k])
    # dx = RN(t s), dr = RN(t): |dx - s dr| <= u (|dx| + s |dr|), u = 2^-8
    s = float(dref.scale(0.25))
    d = (dx.float() - s * dr.float()).abs()
    bound = 2.0 ** -8 * (dx.float().abs() + s * dr.float().abs())
    assert (d[k] <= bound[k] * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("mode", [0, 1], ids=["rms", "layer"])
def test_dropout_add_without_dropout(mode):
    """p = 0: the forward is norm_add_fwd bit for bit and dx = dr."""
    case, ins = _add_case(mode, 65, 1024, 3)
    h, y, rstd, mean, dx, dr, dg, db = _run_add(ins, case, mode, 0.0)
    x, r, g, b, dy, dh = [None if t is None else t.cuda() for t in ins]
    want = gb.norm_add_fwd(x, r, g, b, case.eps, mode)
    for u, v in zip((h, y, rstd, mean), want):
        assert u is v is None or torch.equal(u, v)
    assert torch.equal(dx, dr)
    d2, dg2, db2 = gb.norm_add_bwd(dy, dh, h, g, rstd, mean, mode)
    assert torch.equal(dr, d2) and torch.equal(dg, dg2)


def test_dropout_add_deterministic_streams_and_graph():
    case, ins = _add_case(1, 333, 2048, 9)
    a = _run_add(ins, case, 1, 0.1)
    word = torch.zeros(1, dtype=torch.int64, device="cuda")
    x, r, g, b, dy, dh = [t.cuda() for t in ins]
    ws = torch.empty(gb.norm_dropout_add_bwd_workspace_bytes(333, 2048, 1), dtype=torch.uint8,
                     device="cuda")
    outs = [torch.empty_like(t) for t in a]

    def step():
        rng = dict(p=0.1, seed=SEED, offset=OFF, offset_dev=word)
        gb.norm_dropout_add_fwd(x, r, g, b, case.eps, 1, h=outs[0], y=outs[1], rstd=outs[2],
                                mean=outs[3], **rng)
        gb.norm_dropout_add_bwd(dy, dh, outs[0], g, outs[2], outs[3], 1, dx=outs[4], dr=outs[5],
                                dgamma=outs[6], dbeta=outs[7], workspace=ws, **rng)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    for u, v in zip(outs, a):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for t in outs:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(outs, a):
        assert torch.equal(u, v)
    word.fill_(1)  # another mask on the next replay
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(outs[0], a[0])
    k = dref.keep(x.shape, 0.1, SEED, OFF + 1).cuda()
    assert torch.equal(outs[0][~k], r[~k])
