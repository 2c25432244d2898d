"""Host-side argument checks of the layer operators: every refusal comes before
a device is touched (no compute call runs here)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from _util import lib

    return lib()


def test_fp8_refusals(L):
    raw = L.load()
    assert raw.fp4_fp8_act_scale_bytes(5, 272) == 3 * 8 * 4
    assert raw.fp4_fp8_act_scale_bytes(5, 270) == 0
    assert raw.fp4_quant_act_fp8_b128(16, 16, 16, 4, 24, None) == 2           # K % 16
    assert raw.fp4_quant_act_fp8_b128(None, 16, 16, 4, 32, None) == 1
    assert raw.fp4_quant_act_fp8_b128(16, 24, 16, 4, 32, None) == 3
    assert raw.fp4_quant_act_fp8_b128(None, None, None, 0, 32, None) == 0     # M = 0
    assert raw.fp4_quant_weight_fp8_b128(16, 16, 16, 0, 32, None) == 2        # N = 0
    assert raw.fp4_quant_weight_fp8_b128(16, 16, None, 8, 32, None) == 1
    assert raw.fp4_gemm_fp8_b128(16, 16, 16, 16, None, 16, 4, 12, 32, None) == 2   # N % 8
    assert raw.fp4_gemm_fp8_b128(16, 16, 16, 16, None, 16, 4, 8, 40, None) == 2    # K % 16
    assert raw.fp4_gemm_fp8_b128(16, 16, 16, 16, None, 16, -1, 8, 32, None) == 2
    assert raw.fp4_gemm_fp8_b128(16, 16, None, 16, None, 16, 4, 8, 32, None) == 1
    assert raw.fp4_gemm_fp8_b128(16, 16, 16, 18, None, 16, 4, 8, 32, None) == 3
    assert raw.fp4_gemm_fp8_b128(16, 16, 16, 16, 24, 16, 4, 8, 32, None) == 3
    assert raw.fp4_gemm_fp8_b128(None, None, None, None, None, None, 0, 8, 32, None) == 0
    need = raw.fp4_linear_fp8_b128_workspace_size(5, 8, 272)
    assert need == 1536 + 256
    assert raw.fp4_linear_fp8_b128_workspace_size(0, 8, 272) == 0
    assert raw.fp4_linear_fp8_b128(16, 16, 16, None, 16, 5, 8, 272, 256, need - 1, None) == 1
    assert raw.fp4_linear_fp8_b128(16, 16, 16, None, 16, 5, 8, 272, None, need, None) == 1
    assert raw.fp4_linear_fp8_b128(16, 16, 16, None, 16, 5, 8, 272, 128, need, None) == 3


def _cache(L, **kw):
    f = dict(k_codes=256, k_scales=256, v_codes=256, v_scales=256, num_pages=4, page_size=16, kv_heads=2, head_dim=64,
             format=1)
    f.update(kw)
    return L.fp4_kv_cache(*(f[n] for n, _ in L.fp4_kv_cache._fields_))


def _rope(L, **kw):
    f = dict(table=256, table_positions=8, rot_dim=64, layout=0, flags=0)
    f.update(kw)
    return L.fp4_rope_params(*(f[n] for n, _ in L.fp4_rope_params._fields_))


BAD_CACHES = [(dict(k_codes=0), 1), (dict(v_scales=0), 1), (dict(format=2), 1), (dict(num_pages=0), 2),
              (dict(page_size=24), 2), (dict(page_size=0), 2), (dict(kv_heads=0), 2), (dict(head_dim=96), 2),
              (dict(k_codes=264), 3), (dict(v_codes=264), 3)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_refusals(L, kw, want):
    raw = L.load()
    c = ctypes.byref(_cache(L, **kw))
    assert raw.fp4_kv_append(c, 16, 16, 1, 128, 64, 128, 64, 16, None, None, None) == want
    assert raw.fp4_kv_read(c, 16, 1, 16, 1, 1, 16, 16, None) == want
    a = _attention(L)
    assert raw.fp4_kv_attention(c, ctypes.byref(a), 256, 1 << 20, None) == want


def test_cache_sizes(L):
    raw = L.load()
    assert raw.fp4_kv_code_bytes(ctypes.byref(_cache(L))) == 4 * 2 * 16 * 64
    assert raw.fp4_kv_code_bytes(ctypes.byref(_cache(L, format=0))) == 4 * 2 * 16 * 32
    assert raw.fp4_kv_scale_bytes(ctypes.byref(_cache(L))) == 4 * 2 * 16 * 2
    assert raw.fp4_kv_code_bytes(None) == 0


def test_append_and_read_refusals(L):
    raw = L.load()
    c = ctypes.byref(_cache(L))
    ok = (16, 16, 1, 128, 64, 128, 64, 16)
    assert raw.fp4_kv_append(None, *ok, None, None, None) == 1
    assert raw.fp4_kv_append(c, None, 16, 1, 128, 64, 128, 64, 16, None, None, None) == 1
    assert raw.fp4_kv_append(c, 16, 16, 1, 128, 64, 128, 64, None, None, None, None) == 1
    assert raw.fp4_kv_append(c, 16, 16, -1, 128, 64, 128, 64, 16, None, None, None) == 2
    assert raw.fp4_kv_append(c, 16, 16, 1, 124, 64, 128, 64, 16, None, None, None) == 3      # stride % 8
    assert raw.fp4_kv_append(c, 24, 16, 1, 128, 64, 128, 64, 16, None, None, None) == 3
    assert raw.fp4_kv_append(c, None, None, 0, 128, 64, 128, 64, None, None, None, None) == 0
    assert raw.fp4_kv_append(c, *ok, ctypes.byref(_rope(L)), None, None) == 1                # no positions
    assert raw.fp4_kv_append(c, *ok, ctypes.byref(_rope(L, rot_dim=80)), 16, None) == 2      # beyond the head
    assert raw.fp4_kv_read(c, None, 1, 16, 1, 1, 16, 16, None) == 1
    assert raw.fp4_kv_read(c, 16, 0, 16, 1, 1, 16, 16, None) == 2
    assert raw.fp4_kv_read(c, 16, 1, 16, 0, 1, 16, 16, None) == 2
    assert raw.fp4_kv_read(c, 16, 1, 16, 1, 1, 24, 16, None) == 3
    assert raw.fp4_kv_read(c, None, 1, None, 1, 0, None, None, None) == 0


def test_rope_refusals(L):
    raw = L.load()

    def call(r, tokens=2, heads=2, dim=64, x=16, pos=16, st=(128, 64, 128, 64)):
        return raw.fp4_rope(x, 16, pos, ctypes.byref(r) if r else None, tokens, heads, dim, *st, None)

    assert call(None) == 1
    assert call(_rope(L), pos=None) == 1
    assert call(_rope(L), x=None) == 1
    assert call(_rope(L, layout=2)) == 1
    assert call(_rope(L, flags=2)) == 1
    assert call(_rope(L, table=0)) == 1
    assert call(_rope(L, rot_dim=24)) == 2
    assert call(_rope(L, rot_dim=128)) == 2
    assert call(_rope(L, table_positions=0)) == 2
    assert call(_rope(L), dim=72) == 2
    assert call(_rope(L), heads=0) == 2
    assert call(_rope(L), tokens=-1) == 2
    assert call(_rope(L), st=(-8, 64, 128, 64)) == 2
    assert call(_rope(L), st=(128, 60, 128, 64)) == 3
    assert call(_rope(L, table=264)) == 3
    assert call(_rope(L), tokens=0) == 0
    sc = L.fp4_rope_scaling
    for kind, bad in ((sc(3, 1, 0, 1, 1, 1), 1), (sc(1, 0.5, 0, 1, 1, 1), 1), (sc(2, 2, 0, 32, 1, 1), 1),
                      (sc(2, 2, 4096, 1, 2, 1), 1), (sc(2, 2, 4096, 32, 1, 0), 1)):
        assert raw.fp4_rope_table(16, 8, 64, 10000.0, ctypes.byref(kind), None) == bad
    assert raw.fp4_rope_table(16, 0, 64, 10000.0, None, None) == 2
    assert raw.fp4_rope_table(16, 8, 40, 10000.0, None, None) == 2
    assert raw.fp4_rope_table(16, 8, 64, 1.0, None, None) == 1
    assert raw.fp4_rope_table(24, 8, 64, 10000.0, None, None) == 3


def _attention(L, **kw):
    f = dict(q_bf16=16, out_bf16=16, lse=None, q_token_stride=256, q_head_stride=64, out_token_stride=256,
             out_head_stride=64, block_table=16, block_table_stride=4, context_lens=16, q_offsets=16, tree_mask=None,
             mask_words=0, batch=1, tokens=2, q_heads=4, max_draft=2, max_seq_len=20, softmax_scale=0.125)
    f.update(kw)
    return L.fp4_kv_attention_args(*(f[n] for n, _ in L.fp4_kv_attention_args._fields_))


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 2), (dict(batch=65536), 2), (dict(tokens=-1), 2), (dict(q_heads=3), 2), (dict(q_heads=0), 2),
    (dict(max_draft=0), 2), (dict(max_draft=1025), 2), (dict(max_seq_len=0), 2), (dict(max_seq_len=1), 2),
    (dict(block_table_stride=0), 2), (dict(tree_mask=16, mask_words=1, max_draft=33, max_seq_len=64), 2),
    (dict(q_bf16=None), 1), (dict(out_bf16=None), 1), (dict(block_table=None), 1), (dict(context_lens=None), 1),
    (dict(q_offsets=None), 1), (dict(softmax_scale=0.0), 1), (dict(softmax_scale=float("nan")), 1),
    (dict(softmax_scale=float("inf")), 1), (dict(q_bf16=24), 3), (dict(q_head_stride=60), 3),
    (dict(out_token_stride=252), 3), (dict(lse=18), 3), (dict(tree_mask=18, mask_words=1), 3), (dict(tokens=0), 0)])
def test_attention_refusals(L, kw, want):
    raw = L.load()
    a = _attention(L, **kw)
    assert raw.fp4_kv_attention(ctypes.byref(_cache(L)), ctypes.byref(a), 256, 1 << 30, None) == want


def test_attention_workspace(L):
    raw = L.load()
    c = ctypes.byref(_cache(L))
    assert raw.fp4_kv_attention(c, None, 256, 1 << 20, None) == 1
    assert raw.fp4_kv_attention_workspace_size(0, 1, 8, 8, 64, 16, 1) == 0
    need = raw.fp4_kv_attention_workspace_size(1, 2, 4, 2, 64, 1 << 20, 2)
    assert need > 0
    a = _attention(L, max_seq_len=1 << 20)
    assert raw.fp4_kv_attention(c, ctypes.byref(a), 256, need - 1, None) == 1
    assert raw.fp4_kv_attention(c, ctypes.byref(a), None, need, None) == 1
    assert raw.fp4_kv_attention(c, ctypes.byref(a), 128, need, None) == 3
