"""Attention whose device waits run out: with a test hook the first CTA never
multiplies with the values, so every wait for that product expires.  The call
ends and reports it, the units of that CTA are not written, the others are as
ever, and the next call is right."""
import numpy as np
import pytest

import _layer_ref as R
from _util import lib
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


# units of one, two, three and more tiles, runs of several units, and contexts cut over CTAs
@pytest.mark.parametrize("lens", [[(3, 5)], [(200, 4), (0, 2)], [(380, 8)], [(100, 8), (300, 3), (0, 1)] * 40,
                                  [(9000, 8), (1, 1)], [(600, 2)] * 100],
                         ids=lambda l: "%d-%d" % (len(l), l[0][0]))
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_expired_waits_end_the_call(L, lens, group, fmt):
    import torch

    lens = [(c, min(n, 32 // group) if group == 4 else n) for c, n in lens]
    lens[0] = (lens[0][0], 8 if group == 4 else 9)        # 32 rows: the tile kernel; 72: the row kernel
    p = Problem(lens, 2, group, 128, 16, fmt, tree=False, seed=len(lens))
    good, good_lse = p.run(L)
    L.fp4_debug_set_wait_fault(2_000_000, 1)
    try:
        out, _ = p.run(L, out=torch.full_like(p.q.cuda(), 7.0))
        status = L.fp4_get_device_status()
    finally:
        L.fp4_debug_set_wait_fault(0, 0)
    assert status == L.FP4_ERR_TIMEOUT
    assert L.fp4_get_device_status() == 0
    if max(c + n for c, n in lens) <= 512:                # units are not cut: no partial results
        rows = (out == 7.0).all(-1)
        assert rows[0, 0]                                 # the first unit is the first CTA's
        assert np.array_equal(out[~rows], good[~rows])
    again, again_lse = p.run(L)
    assert np.array_equal(again, good) and np.array_equal(again_lse, good_lse)
