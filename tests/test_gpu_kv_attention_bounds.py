"""Attention with lengths that the host's bounds do not hold, or only just.

A sequence with more drafted tokens than max_draft: the tokens up to the bound
are computed as ever (bounds of test_gpu_kv_attention), those past it give NaN
in the output and the log-sum, whatever the output and the workspace held."""
import numpy as np
import pytest

import _layer_ref as R
from _util import bf16_bits_host, bf16_bits_to_f64, dev, host, lib
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def _attend(L, p, max_draft, max_seq, lens=None):
    """The problem's call with bounds of the caller's, on buffers that hold plausible numbers."""
    import torch

    arrays = [dev(a) for a in p.arrays]
    cache = L.kv_cache(*arrays, p.page, p.fmt)
    q = p.q.cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((p.total, p.heads * p.group), 7.0, device="cuda")
    need = L.fp4_kv_attention_workspace_size(len(p.lens), p.total, p.heads * p.group, p.heads, p.dim, max_seq, max_draft)
    ws = torch.ones(max(need, 4) // 4, device="cuda")
    ctx = dev(np.array([c for c, _ in p.lens], np.int32))
    L.fp4_kv_attention(cache, q, out, dev(p.table), ctx, dev(p.cu), max_seq, max_draft, ws,
                       tree_mask=dev(p.mask_bits().view(np.int32)) if p.tree else None, lse=lse, softmax_scale=p.scale)
    assert L.fp4_get_device_status() == 0
    return bf16_bits_to_f64(bf16_bits_host(out)), host(lse).astype(np.float64)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
# heads of a key head, and the bound: kernels of 4, 8, 16, 32 and 128 rows and of two row tiles
@pytest.mark.parametrize("group,bound", [(1, 3), (4, 1), (3, 2), (4, 4), (4, 7), (1, 20), (4, 9), (8, 20)])
@pytest.mark.parametrize("ctx,max_seq", [(40, 400), (2300, 4000)])
@pytest.mark.parametrize("tree", [False, True])
def test_tokens_past_the_bound_are_nan(L, fmt, group, bound, ctx, max_seq, tree):
    over = bound + 5 if bound < 16 else bound + 41
    p = Problem([(ctx, over), (11, bound), (ctx // 2, bound + 1), (3, 0)], 2, group, 64, 16, fmt, tree, seed=bound + group)
    out, lse = _attend(L, p, bound, max_seq)
    past = np.zeros(p.total, bool)
    for b, (_, n) in enumerate(p.lens):
        past[p.cu[b] + bound:p.cu[b] + max(n, bound)] = True
    assert past.any() and np.isnan(out[past]).all() and np.isnan(lse[past]).all()
    # the tokens up to the bound see what they saw
    whole, wl = p.run(L)
    p.check(np.where(past[:, None, None], whole, out), np.where(past[:, None], wl, lse))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("group,draft", [(4, 1), (4, 4), (4, 8), (4, 31)])
def test_scores_far_below_zero_still_count(L, fmt, group, draft):
    """Equal keys, every score -2^103: the softmax is uniform over what a row sees,
    however far below zero the scores lie."""
    import torch

    p = Problem([(200, draft), (0, draft)], 2, group, 64, 16, fmt, tree=False, seed=draft)
    p.arrays[0][:] = 0x38 if fmt == R.MXFP8 else 0x22      # ones
    p.arrays[1][:] = 127 + 50
    p.q = torch.full_like(p.q, -2.0 ** 50)
    score = -p.scale * 64 * 2.0 ** 100
    out, lse = p.run(L)
    for b, (ctx, n) in enumerate(p.lens):
        t = np.arange(ctx + n)
        pg, sl = p.table[b, t // p.page], t % p.page
        v = R.mx_values(R.unpack(p.arrays[2][pg, :, sl], fmt), p.arrays[3][pg, :, sl], fmt)
        for i in range(n):
            ref = v[:ctx + i + 1].mean(0).repeat(group, 0)
            mag = np.abs(v[:ctx + i + 1]).mean(0).repeat(group, 0)
            bound = 1.01 * 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -19) * mag + (ctx + n) * 2.0 ** -61
            assert np.all(np.abs(out[p.cu[b] + i] - ref) <= bound)
            assert np.all(np.abs(lse[p.cu[b] + i] - score) <= (64 + 8) * 2.0 ** -23 * -score)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("group", [1, 4])
def test_drafted_tokens_beyond_the_table_are_not_seen(L, fmt, group):
    """20 drafted tokens over a table row of one page of 16: every row sees the tokens
    that the table names, as if the cache ended there."""
    p = Problem([(0, 20)], 2, group, 64, 16, fmt, tree=False, seed=group)
    p.table = p.table[:, :1]
    out, lse = _attend(L, p, 20, 20)
    t = np.arange(16)
    k, v = (R.mx_values(R.unpack(p.arrays[2 * i][p.table[0, 0], :, t], fmt), p.arrays[2 * i + 1][p.table[0, 0], :, t], fmt)
            for i in range(2))
    q, sees = p.q.double().numpy(), t[None] <= np.arange(20)[:, None]
    for h in range(2 * group):
        ref, rl, absv, mag = R.attend(q[:, h], k[:, h // group], v[:, h // group], sees, p.scale)
        e = (64 + 8) * 2.0 ** -23 * mag
        bound = 1.01 * 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -19) * absv + 16 * 2.0 ** -61
        assert np.all(np.abs(out[:, h] - ref) <= bound)
        assert np.all(np.abs(lse[:, h] - rl) <= e + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_many_heads_with_the_largest_bound(L, fmt):
    """768 query heads and a bound of 1024 drafted tokens: the bounds' product is no limit."""
    p = Problem([(40, 2), (3, 1)], 8, 96, 64, 16, fmt, tree=False, seed=3)
    p.check(*_attend(L, p, 1024, 2048))
