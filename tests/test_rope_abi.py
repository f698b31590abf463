"""norm_rope_fwd / norm_rope_bwd through the C ABI: what the tensor binding never
passes."""
import ctypes

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

vp = lambda t: t.data_ptr()  # noqa: E731


def _call(T, H, D, odd, dtype, inter, backward, seed=0):
    """One call on dense heads; `odd` is the stride given for a single token or
    head.  Returns the outputs."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    x, dy, gamma = rnd(T, H, D), rnd(T, H, D), rnd(D)
    pos = torch.arange(5, 5 + T).cuda()
    inv = torch.tensor([0.9 ** i for i in range(D // 2)], dtype=torch.float64).cuda()
    out, dgamma = torch.empty_like(x), torch.empty(D, device="cuda")
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[dtype]

    def heads(t):
        return ctypes.byref(gb._binding.Heads(vp(t), H * D if T > 1 else odd, D if H > 1 else odd))

    rot = (T, H, 0, D, D, vp(pos), 64, 0, vp(inv), None, 1, inter)
    s = torch.cuda.current_stream().cuda_stream
    if backward:
        n = gb.norm_rope_bwd_workspace_bytes(T, H, 0, D)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        st = gb.lib().norm_rope_bwd(heads(dy), None, heads(x), None, *rot, vp(gamma), None, 1e-6, 0,
                                    code, heads(out), None, vp(dgamma), None, None, None, vp(ws), n, s)
    else:
        dgamma.zero_()
        st = gb.lib().norm_rope_fwd(heads(x), None, *rot, vp(gamma), None, None, None, 1e-6, 0, code,
                                    heads(out), None, s)
    assert st == 0
    torch.cuda.synchronize()
    return out, dgamma


def test_rows_that_overlap_far_apart_are_refused():
    """Token and head strides of 2^40: token 1 of head 0 is token 0 of head 1,
    though (T - 1) * stride is 2^64."""
    def call(T, H, ts, hs):
        far, near = gb._binding.Heads(256, ts, hs), gb._binding.Heads(256, 16 * H, 16)
        return gb.lib().norm_rope_fwd(ctypes.byref(near), None, T, H, 0, 16, 16, 256, 64, 0, 256,
                                      None, 1, 0, None, None, None, None, 1e-6, 0, 0,
                                      ctypes.byref(far), None, None)

    wide = 1 << 40
    assert call((1 << 24) + 1, 3, wide, wide) == 2
    assert call(1 << 31, 3, wide, wide) == 2
    assert call(4, 3, 20, 75) == 2             # tokens 20 apart reach to 76
    if not torch.cuda.is_available():          # (on a GPU these would run)
        assert call(4, 3, 20, 76) == 7
        assert call(1 << 31, 2, 16, 16 << 31) == 7
        assert call(1 << 31, 65536, wide, 16) == 7


@pytest.mark.gpu
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 5), (5, 1), (1, 1), (1, 300)])
def test_the_stride_of_a_single_token_or_head_is_not_used(T, H, dtype, inter, backward):
    """Lanes beyond the last row step by the strides too: by none that leaves an
    address unaligned."""
    for D in (128, 80):
        want = _call(T, H, D, 0, dtype, inter, backward)
        for odd in (3, 1 << 40):
            for a, b in zip(_call(T, H, D, odd, dtype, inter, backward), want):
                assert torch.equal(a, b)
