"""The attention block's whole prompts and its normed heads: the calls that it makes,
one by one, give the same bits; steps go on from what a prompt left in the cache; and
attention over prompts whose device waits run out ends and says so."""
import numpy as np
import pytest

import _layer_ref as R
from _util import dev, lib
from test_gpu_attention_block import D, HIDDEN, HKV, HQ, PAGE, _step
from test_gpu_prompt_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def _block(L, fmt, normed, max_tokens=700, max_batch=4, max_seq_len=800, pages=160, max_draft=8):
    import torch

    from nvfp4_mxfp4_w4a4_gb300 import attention_block as A

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = lambda n, k: (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).bfloat16()  # noqa: E731
    table = torch.empty(max_seq_len, D, device="cuda")
    L.fp4_rope_table(table, max_seq_len, D, 10000.0)
    cache = A.allocate_cache(pages, PAGE, HKV, D, fmt)
    norm = {}
    if normed:
        norm = {n: (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() for n in ("q_norm", "k_norm")}
    return A.AttentionBlock(A.Fp8Linear.from_bf16(w((HQ + 2 * HKV) * D, HIDDEN)), A.Fp8Linear.from_bf16(w(HIDDEN, HQ * D)),
                            cache, L.rope_params(table, D), HQ, max_tokens, max_batch, max_seq_len, max_draft, prompts=True,
                            **norm)


def _inputs(lens, seed=0):
    import torch

    r = np.random.default_rng(seed)
    pages = [-(-(n + 8) // PAGE) for n in lens]
    order = r.permutation(160).astype(np.int32)
    table = np.zeros((len(lens), max(pages)), np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    seq = np.repeat(np.arange(len(lens)), lens)
    slots = table[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    x = torch.randn(len(pos), HIDDEN, generator=g, device="cuda").bfloat16()
    return x, dev(pos), dev(slots), dev(cu), table


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_prompt_is_its_calls(L, fmt, normed):
    import torch

    block = _block(L, fmt, normed)
    lens = [300, 1, 0, 170]
    x, pos, slots, cu, table = _inputs(lens)
    out = block.prompt(x, pos, slots, cu).clone()
    cached = [t.clone() for t in block.cache.tensors]
    other = _block(L, fmt, normed)
    T = x.shape[0]
    qkv = torch.empty(T, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(block.qkv.workspace_size(T), block.o.workspace_size(T)), dtype=torch.uint8, device="cuda")
    block.qkv(x, qkv, ws)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    qr, kr = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, HKV, D, dtype=torch.bfloat16, device="cuda")
    if normed:
        L.fp4_qk_norm_rope(q, k, qr, kr, block.q_norm, block.k_norm, 1e-6, pos, block.rope)
    else:
        L.fp4_rope(q, qr, pos, block.rope)
        L.fp4_rope(k, kr, pos, block.rope)
    L.fp4_kv_append(other.cache, kr, v, slots)
    a, want = torch.empty_like(qr), torch.empty_like(out)
    aws = torch.empty(max(L.fp4_prompt_attention_workspace_size(4, T, T, HQ, HKV, D), 1), dtype=torch.uint8, device="cuda")
    L.fp4_prompt_attention(qr, kr, v, a, cu, None, aws)
    block.o(a.flatten(1), want, ws)
    assert torch.equal(out, want)
    for mine, theirs in zip(cached, other.cache.tensors):
        assert torch.equal(mine, theirs)
    # the same from a graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = block.prompt(x, pos, slots, cu)
    again.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    assert L.fp4_get_device_status() == 0


@pytest.mark.parametrize("normed", [False, True])
def test_steps_go_on_from_a_prompt(L, normed):
    """A prompt at once and in pieces of steps leave the same cache where the heads are
    normed (both quantize the same bf16 keys), and the steps after it are the same.
    Without norms a step rotates and quantizes keys in one go and a prompt by way of
    bf16: each is off by half a step of E4M3, 2^-4 of the element or 2^-10 of the scale,
    and the prompt's by bf16's 2^-8 too."""
    import torch

    lens = [40, 9]
    x, pos, slots, cu, table = _inputs(lens, 3)
    whole, pieces = _block(L, R.MXFP8, normed), _block(L, R.MXFP8, normed)
    whole.prompt(x, pos, slots, cu)
    starts = [0, 40]
    for at in range(0, 40, 8):
        seqs = [(min(at, n), max(min(8, n - at), 0)) for n in lens]
        part = torch.cat([x[s + c:s + c + n] for s, (c, n) in zip(starts, seqs)])
        _step(pieces, part, seqs, table)
    a, b = ([t.cpu().numpy() for t in block.cache.tensors] for block in (whole, pieces))
    for i in range(0 if normed else 2, 4):
        assert np.array_equal(a[i], b[i])
    ka, kb = (R.mx_values(t[0], t[1], R.MXFP8) for t in (a, b))
    scale = 2.0 ** (np.maximum(a[1], b[1]).astype(np.float64) - 127).repeat(32, -1)
    assert (np.abs(ka - kb) <= (2 * 2.0 ** -4 + 2.0 ** -8) * 1.07 * np.maximum(np.abs(ka), np.abs(kb)) + 2 * 2.0 ** -10 * scale).all()
    fresh = torch.randn(2, HIDDEN, device="cuda").bfloat16()
    after = [_step(block, fresh, [(n, 1) for n in lens], table)[0] for block in (whole, pieces)]
    if normed:
        assert torch.equal(*after)
    assert L.fp4_get_device_status() == 0


def test_a_normed_step_is_its_calls(L):
    import torch

    block, plain = _block(L, R.MXFP8, True), _block(L, R.MXFP8, False)
    x, pos, slots, cu, table = _inputs([5, 3], 7)
    out, _, _ = _step(block, x, [(0, 5), (0, 3)], table)
    T = 8
    qkv = torch.empty(T, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(block.qkv.workspace_size(T), block.o.workspace_size(T)), dtype=torch.uint8, device="cuda")
    block.qkv(x, qkv, ws)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    L.fp4_qk_norm_rope(q, k, q, k, block.q_norm, block.k_norm, 1e-6, pos, block.rope)
    L.fp4_kv_append(plain.cache, k, v, slots)
    a, want = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(out)
    L.fp4_kv_attention(plain.cache, q, a, dev(table), dev(np.zeros(2, np.int32)), cu, block.max_seq_len, block.max_draft, block.attention_ws)
    block.o(a.flatten(1), want, ws)
    assert torch.equal(out, want)


def test_prompt_refusals(L):
    import torch

    block = _block(L, R.MXFP8, False, max_tokens=16, max_batch=2)
    x, pos, slots, cu, _ = _inputs([17])
    with pytest.raises(ValueError):
        block.prompt(x, pos, slots, cu)
    x, pos, slots, cu, _ = _inputs([3, 3, 3])
    with pytest.raises(ValueError):
        block.prompt(x, pos, slots, cu)
    block.prompt_ws = None
    with pytest.raises(ValueError):
        block.prompt(x[:3], pos[:3], slots[:3], cu[:2].contiguous())
    from nvfp4_mxfp4_w4a4_gb300 import attention_block as A

    with pytest.raises(ValueError):
        A.AttentionBlock(block.qkv, block.o, block.cache, block.rope, HQ, 16, 2, 32, 1, q_norm=torch.ones(D, device="cuda").bfloat16())


# units that are dealt out whole, and units cut over CTAs
@pytest.mark.parametrize("lens", [[(3, 3)], [(200, 200), (5, 5)], [(100, 100)] * 60, [(3000, 3000), (1, 1)]])
@pytest.mark.parametrize("dim", [64, 128])
def test_expired_waits_end_the_call(L, lens, dim):
    """With a test hook the first CTA leaves out its products with the values: its waits
    expire, the call ends and reports it, what that CTA would have written is not written
    where units are whole, and the next call is right."""
    import torch

    p = Problem(lens, 2, 2, dim, seed=len(lens))
    ws = p.workspace(L)
    p.run(L, ws=ws)
    p.check()
    good = p.out.clone()
    p.out.fill_(7.0)
    L.fp4_debug_set_wait_fault(2_000_000, 1)
    try:
        p.run(L, ws=ws)
        status = L.fp4_get_device_status()
    finally:
        L.fp4_debug_set_wait_fault(0, 0)
    assert status == L.FP4_ERR_TIMEOUT
    assert L.fp4_get_device_status() == 0
    if lens[0][0] <= 1024:
        rows = (p.out == 7.0).all(-1)
        assert rows[0, 0]
        assert torch.equal(p.out[~rows], good[~rows])
    p.run(L, ws=ws)
    assert torch.equal(p.out, good)
