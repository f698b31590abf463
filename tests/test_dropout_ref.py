"""The dropout reference against the published known answers of
Philox4x32-10, and its mask's frequency."""
import numpy as np
import pytest

import dropout_ref as dr


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(ctr, key, want):
    got = dr.philox(np.array([ctr], np.uint64), key)
    assert tuple(int(v) for v in got[0]) == want


def test_blocks_and_frequency():
    n = 1 << 20
    h = dr.halves(n, seed=(7 << 32) | 5, offset=(1 << 40) + 3)
    # a later stretch of the same stream, and the ragged end
    assert np.array_equal(dr.halves(1000, (7 << 32) | 5, (1 << 40) + 3, first=4096), h[4096:5096])
    for p in (0.1, 0.5):
        T = dr.threshold(p)
        got = np.mean(h < T)
        # binomial: 6 standard deviations
        assert abs(got - T / 65536) < 6 * np.sqrt(p * (1 - p) / n)
    assert dr.scale(0.5) == 2 and dr.scale(0.0) == 1
