"""Prompt attention over units that are cut over CTAs: NaN and Inf in their parts; and
offsets out of order, whose calls write nothing outside the tensors."""
import pytest

from _util import lib
from test_gpu_prompt_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [[(1500, 1500), (70, 1400)], [(200, 5000)], [(1300, 1200), (3, 2000)]])
def test_nan_and_inf_in_cut_units(L, lens, dim, causal):
    """NaN and Inf in queries, keys and values reach exactly the queries that see them,
    whichever part of their unit has them: whole tiles, masked ones, both."""
    p = Problem(lens, 2, 2, dim, seed=31)
    nan, inf = float("nan"), float("inf")
    p.k[p.m:], p.v[p.m:] = nan, nan
    m0 = lens[0][1]
    for back, head, at, x in ((1, 0, 3, nan), (40, 1, 5, inf), (41, 1, 6, -inf), (20, 1, 6, inf), (700, 0, 9, inf),
                              (701, 0, 10, -inf), (130, 0, 10, inf), (m0 - 7, 1, 20, -inf), (500, 1, 33, nan)):
        p.v[m0 - back, head, at] = x
    p.k[m0 - 3, 0, 7] = nan
    p.k[m0 - 600, 1, 8] = nan
    p.q[2, 1, 0] = nan
    p.q[lens[0][0] - 5, 3, 1] = nan
    if len(lens) > 1:
        m1 = m0 + lens[1][1]
        p.v[m1 - 1, 1] = inf
        p.v[m1 - 900, 0, 9] = nan
        p.v[m1 - 50, 1, 11] = -inf
    p.run(L, causal)
    p.check(causal)


# (few keys: whole units; many: units cut over CTAs)
@pytest.mark.parametrize("tokens,keys", [(100, 100), (700, 3000)])
@pytest.mark.parametrize("causal", [True, False])
def test_offsets_out_of_order_write_nothing_outside(L, tokens, keys, causal):
    import torch

    p = Problem([(tokens, keys)], 2, 2, 64, seed=7, extra=0)
    edge = 300
    out = torch.full((tokens + 2 * edge, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tokens + 2 * edge, 4), 7.0, dtype=torch.float32, device="cuda")
    p.out, p.lse = out[edge:edge + tokens], lse[edge:edge + tokens]
    big = 2 ** 31 - 1
    for cu, cu_k in (([0, 200, -5, 60, 2 ** 30], [0, big, 50, -7, 90]), ([-9, big, -big - 1, 5, 5], [keys, 0, keys, 0, big]),
                     ([tokens, tokens, 0, tokens, 1], [-3, -2, -1, keys, keys]), ([5, 50, 7, big, big], [0, 0, 0, 0, 0])):
        p.cu, p.cu_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, cu_k))
        p.lens = [(1, 1)] * 4
        p.run(L, causal)
        torch.cuda.synchronize()
        assert L.fp4_get_device_status() == 0
        for x in (out, lse):
            assert (x[:edge] == 7.0).all() and (x[edge + tokens:] == 7.0).all()
