"""The attention block's serving steps: the FP8 linear layer, rotary positions,
the cache and attention working on each other's results."""
import numpy as np
import pytest

import _layer_ref as R
from _util import bf16_bits_host, bf16_bits_to_f64, dev, host, lib

pytestmark = pytest.mark.gpu

HIDDEN, HQ, HKV, D, PAGE = 512, 8, 2, 64, 16


@pytest.fixture(scope="module")
def L():
    return lib()


def _block(L, fmt, max_tokens=64, max_batch=4, max_seq_len=160, max_draft=64, pages=48):
    import torch

    from nvfp4_mxfp4_w4a4_gb300 import attention_block as A

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = lambda n, k: (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).bfloat16()  # noqa: E731
    table = torch.empty(max_seq_len, D, device="cuda")
    L.fp4_rope_table(table, max_seq_len, D, 10000.0)
    cache = A.allocate_cache(pages, PAGE, HKV, D, fmt)
    return A.AttentionBlock(A.Fp8Linear.from_bf16(w((HQ + 2 * HKV) * D, HIDDEN)), A.Fp8Linear.from_bf16(w(HIDDEN, HQ * D)),
                            cache, L.rope_params(table, D), HQ, max_tokens, max_batch, max_seq_len, max_draft)


def _step(block, x, seqs, table, mask=None):
    """seqs: (context, new tokens) of each sequence, whose pages are rows of table."""
    pos = np.concatenate([np.arange(c, c + n) for c, n in seqs]).astype(np.int32)
    seq = np.repeat(np.arange(len(seqs)), [n for _, n in seqs])
    slots = table[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
    cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
    ctx = np.array([c for c, _ in seqs], np.int32)
    out = block.step(x, dev(pos), dev(slots), dev(table), dev(ctx), dev(cu), None if mask is None else dev(mask))
    return out.clone(), pos, seq


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_each_stage_works_on_the_one_before(L, fmt):
    import torch

    block = _block(L, fmt)
    r = np.random.default_rng(0)
    table = r.permutation(48).astype(np.int32)[:40].reshape(4, 10)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    filled = [0, 0, 0]
    for news in ([40, 9, 3], [1, 1, 1], [5, 0, 8]):
        seqs = list(zip(filled, news))
        x = torch.randn(sum(news), HIDDEN, generator=g, device="cuda").bfloat16()
        out, pos, seq = _step(block, x, seqs, table[:3])
        assert L.fp4_get_device_status() == 0
        T = len(pos)
        # rotated queries in place, and the attention of what the cache now holds
        q = bf16_bits_to_f64(bf16_bits_host(block.projected[:T]))[:, :HQ * D].reshape(T, HQ, D)
        got = bf16_bits_to_f64(bf16_bits_host(block.attended[:T])).reshape(T, HQ, D)
        kv = [R.mx_values(R.unpack(host(block.cache.tensors[2 * i]), fmt), host(block.cache.tensors[2 * i + 1]), fmt)
              for i in range(2)]
        for b, (c, n) in enumerate(seqs):
            if n == 0:
                continue
            t = np.arange(c + n)
            k, v = (a[table[b, t // PAGE], :, t % PAGE] for a in kv)
            sees = t[None] <= (c + np.arange(n))[:, None]
            rows = np.flatnonzero(seq == b)
            for h in range(HQ):
                ref, _, absv, mag = R.attend(q[rows, h], k[:, h // 4], v[:, h // 4], sees, D ** -0.5)
                e = (D + 8) * 2.0 ** -23 * mag[:, None]
                bound = 1.01 * 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e + 2.0 ** -19) * absv + (c + n) * 2.0 ** -61
                assert np.all(np.abs(got[rows, h] - ref) <= bound)
        # the output projection of that
        a = np.ascontiguousarray(got.reshape(T, -1))
        codes, scales = R.fp8_quantize(a, 1)
        av, wv = R.fp8_values(codes, scales, 1), R.fp8_values(host(block.o.codes), host(block.o.scales), 128)
        ref, absum = av @ wv.T, np.abs(av) @ np.abs(wv).T
        err = np.abs(bf16_bits_to_f64(bf16_bits_host(out)) - ref)
        assert np.all(err <= 1.01 * 2.0 ** -8 * np.abs(ref) + (128 + 4 + 8) * 2.0 ** -23 * absum)
        filled = [c + n for c, n in seqs]


def test_token_by_token_fills_the_cache_like_a_chunk(L):
    """A chunk of tokens and the same tokens one at a time leave the same cache: the
    projections of a row do not depend on the batch it is in beyond their rounding,
    so codes may differ only where a projection's last bit does."""
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(24, HIDDEN, generator=g, device="cuda").bfloat16()
    table = np.arange(10, dtype=np.int32)[None]
    chunk, single = _block(L, R.MXFP8), _block(L, R.MXFP8)
    whole, _, _ = _step(chunk, x, [(0, 24)], table)
    parts = torch.cat([_step(single, x[i:i + 1], [(i, 1)], table)[0] for i in range(24)])
    for a, b in zip(chunk.cache.tensors, single.cache.tensors):
        assert (host(a) != host(b)).mean() <= 0.01
    a, b = (bf16_bits_to_f64(bf16_bits_host(t)) for t in (whole, parts))
    assert np.linalg.norm(a - b) <= 0.02 * np.linalg.norm(b)


def test_a_tree_gives_each_branch_its_own_result(L):
    """Two branches drafted together (siblings masked from each other) against each
    branch drafted alone, on the same context."""
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    ctx = torch.randn(37, HIDDEN, generator=g, device="cuda").bfloat16()
    draft = torch.randn(4, HIDDEN, generator=g, device="cuda").bfloat16()    # branches (0, 1) and (2, 3)
    table = np.arange(10, dtype=np.int32)[None]
    mask = np.array([[0b0001, 0], [0b0011, 0], [0b0100, 0], [0b1100, 0]], np.int32)
    block = _block(L, R.MXFP8)
    _step(block, ctx, [(0, 37)], table)
    pos = np.array([37, 38, 37, 38], np.int32)
    at = 37 + np.arange(4)
    slots = table[0, at // PAGE].astype(np.int64) * PAGE + at % PAGE
    i32 = lambda *v: dev(np.array(v, np.int32))  # noqa: E731
    both = block.step(draft, dev(pos), dev(slots), dev(table), i32(37), i32(0, 4), dev(mask)).clone()
    for rows in ([0, 1], [2, 3]):
        alone, _, _ = _step(block, draft[rows], [(37, 2)], table)
        a, b = (bf16_bits_to_f64(bf16_bits_host(t)) for t in (both[rows], alone))
        assert np.linalg.norm(a - b) <= 0.02 * np.linalg.norm(b)


def test_more_tokens_than_planned_are_refused(L):
    import torch

    block = _block(L, R.MXFP8, max_tokens=4)
    x = torch.zeros(5, HIDDEN, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        _step(block, x, [(0, 5)], np.arange(10, dtype=np.int32)[None])
