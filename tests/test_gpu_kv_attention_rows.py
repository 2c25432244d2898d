"""Attention where its kernels differ: running references that move again and
again along a context, at row counts of every kernel (up to 4, 8, 16, 32 and
128 rows per unit, and several units), and the precision of few rows.

Bounds: those of test_gpu_kv_attention.  Up to 4 rows a probability enters the
second product as two bf16 parts, of which 2^-16 is lost at most, instead of
its rounding's 2^-8."""
import numpy as np
import pytest

import _layer_ref as R
from _util import lib
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,draft", [(1, 3), (4, 2), (8, 2), (4, 8), (3, 11), (4, 31), (5, 26), (8, 40)])
def test_scores_that_grow_along_the_context(L, fmt, dim, group, draft):
    """The keys' block scales rise by a power of two every 150 tokens, so that the
    largest score passes the reference by 2^8 several times on the way."""
    lens = [(1100, draft), (389, 1), (640, draft)]
    p = Problem(lens, 2, group, dim, 16, fmt, seed=group * draft + dim)
    k_scales = p.arrays[1]
    for b, (ctx, n) in enumerate(lens):
        for t in range(ctx + n):
            k_scales[p.table[b, t // 16], :, t % 16] += np.uint8(t // 150)
    p.check(*p.run(L))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("contexts", [range(120, 136), [0, 1, 127, 128, 255, 256, 257, 383, 384, 385, 511, 512, 513]])
def test_units_of_every_parity(L, fmt, contexts):
    """Many units per CTA whose tile counts differ: even and odd tiles belong to
    different warps, and a unit starts where the one before it ended."""
    p = Problem([(c, 1 + c % 13) for c in contexts] * 3, 4, 6, 64, 32, fmt, seed=3)
    p.check(*p.run(L))
    p.check(*p.run(L, max_seq=4096))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("group,draft", [(1, 1), (4, 1), (2, 2), (1, 3)])
def test_few_rows_keep_their_probabilities(L, fmt, group, draft):
    lens = [(503, draft), (3, draft), (1500, draft)]
    p = Problem(lens, 2, group, 128, 16, fmt, seed=group + draft)
    out, _ = p.run(L)
    q = p.q.double().numpy()
    for b, (ctx, n) in enumerate(lens):
        t = np.arange(ctx + n)
        pg, sl = p.table[b, t // p.page], t % p.page
        k, v = (R.mx_values(R.unpack(p.arrays[2 * i][pg, :, sl], fmt), p.arrays[2 * i + 1][pg, :, sl], fmt)
                for i in range(2))
        sees = np.concatenate((np.ones((n, ctx), bool), p.sees[b]), 1)
        for h in range(p.heads * group):
            kk, vv, qq = k[:, h // group], v[:, h // group], q[p.cu[b]:p.cu[b] + n, h]
            s = np.where(sees, p.scale * qq @ kk.T, -np.inf)
            e = (p.dim + 8) * 2.0 ** -23 * (p.scale * np.abs(qq) @ np.abs(kk).T).max()
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            ref = w @ vv
            bound = 1.01 * 2.0 ** -8 * np.abs(ref) + (2.0 ** -16 + 2 * e + 2.0 ** -19) * (w @ np.abs(vv)) + len(t) * 2.0 ** -61
            assert (np.abs(out[p.cu[b]:p.cu[b] + n, h] - ref) <= bound).all()
