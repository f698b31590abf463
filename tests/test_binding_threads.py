"""The native binding lets other Python threads run while a call waits: a
launch on a full queue waits for the GPU, and that must not stop them."""
import threading
import time

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb

pytestmark = pytest.mark.gpu


def _calls():
    x = torch.randn(2, 8, 64, device="cuda").bfloat16()
    rows = x.view(16, 64)
    g, b = torch.ones_like(x[0, 0]), torch.zeros_like(x[0, 0])
    rng = dict(p=0.1, seed=1)
    y, rstd, mean = gb.norm_group_fwd(x, g, b, 4)
    h, _, rs, mu = gb.norm_dropout_add_fwd(rows, rows, g, b, 1e-5, gb.LAYER, **rng)
    return {
        "dropout": lambda: gb.norm_dropout(x, **rng),
        "dropout_add_fwd": lambda: gb.norm_dropout_add_fwd(rows, rows, g, b, 1e-5, gb.LAYER, **rng),
        "dropout_add_bwd": lambda: gb.norm_dropout_add_bwd(rows, rows, h, g, rs, mu, gb.LAYER, **rng),
        "group_fwd": lambda: gb.norm_group_fwd(x, g, b, 4),
        "group_bwd": lambda: gb.norm_group_bwd(x, x, g, b, rstd, mean, 4),
    }


def _cycles(seconds):
    """Argument of torch.cuda._sleep for about that long."""
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda._sleep(1000)
    a.record()
    torch.cuda._sleep(10_000_000)
    b.record()
    b.synchronize()
    return int(10_000_000 * seconds * 1e3 / a.elapsed_time(b))


@pytest.mark.parametrize("name", ["dropout", "dropout_add_fwd", "dropout_add_bwd", "group_fwd",
                                  "group_bwd"])
def test_a_launch_that_waits_leaves_other_threads_running(name):
    call = _calls()[name]
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    cycles = _cycles(0.6)
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    t = threading.Thread(target=tick)
    t.start()
    try:
        torch.cuda._sleep(cycles)
        begin = end = 0.0
        for _ in range(6000):  # more than the queue of a stream holds
            begin = time.perf_counter()
            call()
            end = time.perf_counter()
            if end - begin > 0.1:
                break
    finally:
        stop.set()
        t.join()
        torch.cuda.synchronize()
    if end - begin <= 0.1:
        pytest.skip("no launch waited")
    # the longest time without a tick while that launch waited
    at = [begin] + [v for v in ticks if begin < v < end] + [end]
    gap = max(v - u for u, v in zip(at, at[1:]))
    assert gap < 0.5 * (end - begin), f"{gap:.3f} s of {end - begin:.3f} s without another thread"


def test_threads_on_streams_of_their_own():
    """Calls of several threads at once, each on its own stream and shapes."""
    def case(i):
        gen = torch.Generator().manual_seed(i)
        B, S, C = ((2, 60, 64), (1, 20000, 256), (20, 50, 320), (3, 700, 168))[i]
        x = torch.randn(B, S, C, generator=gen).bfloat16().cuda()
        g = torch.randn(C, generator=gen).bfloat16().cuda()
        return x, g

    def step(x, g):
        y, rstd, mean = gb.norm_group_fwd(x, g, None, 4, 1e-5, "silu", p=0.1, seed=2)
        rows = x.view(-1, x.shape[-1])
        grads = gb.norm_group_bwd(x, x, g, None, rstd, mean, 4, "silu", p=0.1, seed=2)
        return (y, rstd, mean, *grads,
                *gb.norm_dropout_add_fwd(rows, rows, g, p=0.1, seed=3)[:3], gb.norm_dropout(x, 0.5, 4))

    cases = [case(i) for i in range(4)]
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = step(*cases[i])
                s.synchronize()
                if not all(torch.equal(u, v) for u, v in zip(got, want[i])):
                    bad.append(i)
                    return

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    assert gb.norm_get_device_error() == 0
