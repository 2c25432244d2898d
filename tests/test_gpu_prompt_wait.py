"""Prompt attention whose waits run out where units are cut over CTAs."""
import pytest

from _util import lib
from test_gpu_prompt_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[(3000, 3000), (1, 1)], [(300, 6000)], [(40, 1500)] * 7])
@pytest.mark.parametrize("dim", [64, 128])
def test_cut_units_without_one_of_their_parts_are_not_written(L, lens, dim, causal):
    """The first CTA leaves out its products with the values: its part of a cut unit is
    missing, so that the unit's rows stay as they were, and all others are right."""
    import torch

    p = Problem(lens, 2, 2, dim, seed=len(lens))
    ws = p.workspace(L)
    p.run(L, causal, ws=ws)
    p.check(causal)
    good = p.out.clone(), p.lse.clone()
    p.out.fill_(7.0)
    p.lse.fill_(7.0)
    ws.fill_(0xFF)  # (as float: NaN; nothing of an earlier call)
    torch.cuda.synchronize()
    L.fp4_debug_set_wait_fault(2_000_000, 1)
    try:
        p.run(L, causal, ws=ws)
        status = L.fp4_get_device_status()
    finally:
        L.fp4_debug_set_wait_fault(0, 0)
    assert status == L.FP4_ERR_TIMEOUT
    assert L.fp4_get_device_status() == 0
    untouched = (p.out == 7.0).all(-1)
    assert untouched[0, 0] and not untouched[:p.n].all()
    assert torch.equal(p.out[~untouched], good[0][~untouched])
    assert torch.equal(p.lse == 7.0, untouched)
    assert torch.equal(p.lse[~untouched], good[1][~untouched])
    p.run(L, causal, ws=ws)
    assert torch.equal(p.out, good[0]) and torch.equal(p.lse, good[1])
