"""How exact the angles of far positions are: the bound that the header states, from
the kernel's integer steps restated (CPU) and from its results (GPU), against exact
rationals with 100 digits of pi."""
import math
import random
import struct
from fractions import Fraction

import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb
import rope_ref as rr

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679,
              10 ** 100)
U64 = 1 << 64


def turns(freq):
    """A frequency as a 64-bit fraction of a turn, in the kernel's steps."""
    bits, = struct.unpack("<Q", struct.pack("<d", freq))
    e = bits >> 52 & 2047
    if e == 0:
        return 0
    p = (bits & (1 << 52) - 1 | 1 << 52) * 0xa2f9836e4e44152a
    s = 1077 - e
    f = 0 if s >= 128 or s <= 0 else p >> s
    return (-f if bits >> 63 else f) % U64


def exact_turn(pos, freq):
    return pos * Fraction(freq) / (2 * PI)


def off(turn, want):
    """Distance on the circle, in turns."""
    d = (turn - want) % 1
    return float(min(d, 1 - d))


def bound(pos, freq):
    return abs(pos) * (2.0 ** -64 + abs(freq) * 2.0 ** -72)


def test_the_stated_bound_holds():
    rng = random.Random(1)
    worst = 0.0
    for _ in range(4000):
        freq = rng.choice([-1, 1]) * 2.0 ** rng.uniform(-60, 52.9)
        pos = rng.choice([-1, 1]) * int(2.0 ** rng.uniform(0, 63))
        b = bound(pos, freq)
        d = off(Fraction(pos * turns(freq) % U64, U64), exact_turn(pos, freq))
        if b < 0.5:
            worst = max(worst, d / b)
            assert d <= b, (pos, freq)
    assert worst > 0.9  # and is no wider than it has to be
    # within the ranges that the header names: half a step of fp32 below 1
    assert 2 * math.pi * (bound(2 ** 35, 256) + 2.0 ** -32) < 2.0 ** -25


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("top", [2 ** 31, 2 ** 35])
def test_far_positions_against_exact_angles(top, inter):
    """Frequencies of all 53 bits, up to 256.  The angle's 2^-25 radians come to the
    2^-18 of the magnitudes that the arithmetic is allowed."""
    g = torch.Generator().manual_seed(3)
    pos = [top, -top, top - 1, 1 - top, top // 3, 0, 1, -12345678901 % top]
    freq = [256.0 * 0.7 ** i for i in range(64)]
    x = torch.randn(len(pos), 2, 128, generator=g)
    ang = torch.tensor([[float(2 * PI * (exact_turn(p, f) % 1)) for f in freq] for p in pos],
                       dtype=torch.float64)
    y, _ = gb.norm_rope_fwd(x.cuda(), None, torch.tensor(pos).cuda(),
                            torch.tensor(freq, dtype=torch.float64).cuda(), interleaved=inter)
    want, mag = rr.forward(x.double(), ang, inter)
    rr.check(y.cpu(), want, mag, rr.ARITH_Y + 2.0 ** -25, "y")


@pytest.mark.gpu
def test_beyond_the_promised_range_the_error_grows_as_stated():
    for p in (2 ** 40, 2 ** 48, -2 ** 51, 2 ** 58 + 12345):
        freq = [0.9 ** i for i in range(32)]
        x = torch.ones(1, 1, 64)
        y, _ = gb.norm_rope_fwd(x.cuda(), None, torch.tensor([p]).cuda(),
                                torch.tensor(freq, dtype=torch.float64).cuda())
        ang = torch.tensor([[float(2 * PI * (exact_turn(p, f) % 1)) for f in freq]], dtype=torch.float64)
        want, mag = rr.forward(x.double(), ang, False)
        rr.check(y.cpu(), want, mag, rr.ARITH_Y + 2 * math.pi * bound(p, 1.0), "y")
