"""What a query of a prompt does not see leaves its results as they are, bit for bit:
later keys and values of its sequence, however large, and those of other sequences."""
import pytest

from _util import lib
from test_gpu_prompt_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


# sequences whose units stay whole, and one that is cut over CTAs
@pytest.mark.parametrize("n", [400, 2100])
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (3, 64)])
def test_later_keys_leave_earlier_rows_alone(L, n, group, dim):
    """Keys and values from some position on are made large (their scores then pass the
    earlier rows' maxima many times over), then Inf and NaN: rows before it keep their bits."""
    import torch

    p = Problem([(n, n)], 2, group, dim, seed=n + group)
    ws = p.workspace(L)
    p.run(L, ws=ws)
    p.check()
    out, lse = p.out.clone(), p.lse.clone()
    k, v = p.k.clone(), p.v.clone()
    # (second tiles and later ones, where a row has a reference already, in the middle of a warp's rows)
    for at in (137, 203, 251, 333, 391, n - 59):
        for factor in (-512.0, float("inf"), float("nan")):
            p.k.copy_(k)
            p.v.copy_(v)
            p.k[at:] *= factor
            p.v[at:] *= factor
            p.out.fill_(7.0)
            p.lse.fill_(7.0)
            p.run(L, ws=ws)
            assert torch.equal(p.out[:at], out[:at]) and torch.equal(p.lse[:at], lse[:at]), (at, factor)


def test_other_sequences_leave_rows_alone(L):
    """The same for the keys of the sequences before and behind, in tiles that reach into them."""
    import torch

    lens = [(150, 150), (200, 260), (90, 150)]
    p = Problem(lens, 2, 2, 64, seed=21)
    p.run(L)
    p.check()
    out, lse = p.out.clone(), p.lse.clone()
    for factor in (-512.0, float("inf"), float("nan")):
        q = Problem(lens, 2, 2, 64, seed=21)
        for x in (q.k, q.v):
            x[:150] *= factor
            x[410:] *= factor
        q.run(L)
        assert torch.equal(q.out[150:350], out[150:350]) and torch.equal(q.lse[150:350], lse[150:350])
