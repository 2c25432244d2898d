"""The attention block's step with more tokens than its bounds hold."""
import numpy as np
import pytest

import _layer_ref as R
from _util import lib
from test_gpu_attention_block import HIDDEN, _block, _step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def _x(tokens, seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(tokens, HIDDEN, generator=g, device="cuda").bfloat16()


TABLE = np.arange(40, dtype=np.int32).reshape(4, 10)


@pytest.mark.parametrize("seqs", [[(0, 9)], [(0, 8), (0, 9)], [(20, 17), (0, 0)]])
def test_more_tokens_than_drafts_are_refused(L, seqs):
    block = _block(L, R.MXFP8, max_draft=8)
    with pytest.raises(ValueError):
        _step(block, _x(sum(n for _, n in seqs), 0), seqs, TABLE[:len(seqs)])
    _step(block, _x(8 * len(seqs), 0), [(0, 8)] * len(seqs), TABLE[:len(seqs)])


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("max_draft", [1, 4, 8])
def test_one_long_sequence_among_others_is_nan(L, fmt, max_draft):
    """The sum of the tokens does not show it: rows past the bound are NaN, not what
    an earlier step left, and the others are those of a step within the bounds."""
    import torch

    block = _block(L, fmt, max_draft=max_draft)
    x = _x(max_draft + 1, 1)
    _step(block, _x(2 * max_draft, 2), [(0, max_draft)] * 2, TABLE[:2])     # leaves its rows in the buffers
    out, _, _ = _step(block, x, [(0, max_draft + 1), (0, 0)], TABLE[:2])
    assert torch.isnan(out[max_draft:]).all()
    want, _, _ = _step(block, x[:max_draft], [(0, max_draft), (0, 0)], TABLE[:2])
    a, b = out[:max_draft].double(), want.double()
    assert torch.isfinite(a).all() and (a - b).norm() <= 0.02 * b.norm()
