"""Attention at sizes of its own: more sequences than a CTA has threads, pieces of
a prompt with masks of many words, and a block's step inside a CUDA graph.

Bounds: those of test_gpu_kv_attention."""
import numpy as np
import pytest

import _layer_ref as R
from _util import dev, lib
from test_gpu_attention_block import HIDDEN, PAGE, _block
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
# rows of the longest draft: 4, 16, 32 and 48, one for each kernel and two for the first
@pytest.mark.parametrize("group", [1, 4, 8, 12])
@pytest.mark.parametrize("max_seq", [None, 4096])
def test_many_short_sequences(L, fmt, group, max_seq):
    """1300 sequences, of some of which nothing is drafted, among them long ones."""
    r = np.random.default_rng(group)
    lens = [(int(c), int(n)) for c, n in zip(r.integers(0, 40, 1300), r.integers(0, 5, 1300))]
    for i in range(17, 1300, 97):
        lens[i] = (int(r.integers(300, 1500)), int(r.integers(0, 5)))
    lens[-1] = (700, 4)
    p = Problem(lens, 1, group, 64, 16, fmt, seed=group)
    p.check(*p.run(L, max_seq))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens,group", [([(40, 700), (5, 130), (0, 65)], 1), ([(513, 300), (1, 257)], 3), ([(90, 1024)], 1)])
def test_pieces_of_a_prompt(L, fmt, tree, lens, group):
    p = Problem(lens, 1, group, 64, 32, fmt, tree, seed=lens[0][1])
    p.check(*p.run(L))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("max_draft,news", [(1, (1, 1, 1)), (4, (4, 1, 2)), (8, (8, 3, 8)), (64, (40, 1, 23))])
def test_a_step_in_a_graph(L, fmt, max_draft, news):
    """A captured step, replayed on other inputs, gives the bits of the step called."""
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(max_draft)
    T, ctx = sum(news), (30, 0, 77)
    table = np.arange(40, dtype=np.int32).reshape(4, 10)[:3]
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, news)]).astype(np.int32)
    seq = np.repeat(np.arange(3), news)
    slots = table[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
    static = [dev(pos), dev(slots), dev(table), dev(np.array(ctx, np.int32)),
              dev(np.concatenate([[0], np.cumsum(news)]).astype(np.int32))]
    xs = [torch.randn(T, HIDDEN, generator=g, device="cuda").bfloat16() for _ in range(3)]
    x = xs[0].clone()
    captured, called = _block(L, fmt, max_draft=max_draft), _block(L, fmt, max_draft=max_draft)
    captured.step(x, *static)               # the one-time set-up of the kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.step(x, *static)
    for other in xs[1:]:
        x.copy_(other)
        graph.replay()
        want = called.step(other, *static)
        assert torch.equal(out, want) and torch.isfinite(out).all()
        for a, b in zip(captured.cache.tensors, called.cache.tensors):
            assert torch.equal(a, b)
    assert L.fp4_get_device_status() == 0
