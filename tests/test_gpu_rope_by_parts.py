"""Frequencies of the by-parts rotary table at the ends of its ramp: the ramp
runs to the index of the slow end, which may lie past the last frequency
(index rot_dim / 2 - 1), and is only cut at rot_dim - 1."""
import math

import numpy as np
import pytest

from _util import host, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def _frequencies(rot, base, factor, original, fast, slow):
    half = rot // 2
    w = base ** (-np.arange(half) / half)

    def index(turns):
        return half * math.log(original / (2 * math.pi * turns)) / math.log(base)

    low, high = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    i = np.arange(half)
    # where the ends meet the ramp is a step: up to that index nothing is interpolated
    ramp = np.clip((i - low) / (high - low), 0, 1) if high > low else (i > high).astype(float)
    return w * (1 - ramp) + w / factor * ramp, low, high


# the slow end past the last frequency, past the last index, inside, and both ends at index 0
@pytest.mark.parametrize("rot,base,original,fast,slow,ends", [
    (128, 10000.0, 65536, 32.0, 1.0, (40, 65)), (64, 500.0, 1 << 22, 32.0, 1.0, (51, 63)),
    (128, 10000.0, 4096, 32.0, 1.0, (20, 46)), (16, 10000.0, 1000, 300.0, 283.0, (0, 0))])
def test_ends_of_the_ramp(L, rot, base, original, fast, slow, ends):
    import torch

    w, low, high = _frequencies(rot, base, 8.0, original, fast, slow)
    assert (low, high) == ends
    P = 3000
    t = torch.empty(P, rot, device="cuda")
    L.fp4_rope_table(t, P, rot, base, L.FP4_ROPE_BY_PARTS, 8.0, original, fast, slow, 1.0)
    a = np.arange(P)[:, None] * w
    # one float32 rounding; the angle (up to 3000) carries a few 64-bit roundings
    assert np.max(np.abs(host(t) - np.concatenate((np.cos(a), np.sin(a)), 1))) <= 2.0 ** -24 + 1e-11
