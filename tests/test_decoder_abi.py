"""Host-side argument checks of head norms, prompt attention, 4-bit matrix-vector
products and expert dispatch, in the library and in the binding: every refusal
comes before a device is touched (no compute call runs here)."""
import ctypes

import pytest
import torch

from test_layer_binding import F32, I32, I64, U8, L, _host, _refused, _rope, _z  # noqa: F401
from nvfp4_mxfp4_w4a4_gb300 import fp4lin


@pytest.fixture(scope="module")
def raw():
    from _util import lib

    return lib().load()


# -------------------------------------------------------------- the library


def _fill(kind, f, kw):
    f.update(kw)
    return ctypes.byref(kind(*(f[n] for n, _ in kind._fields_)))


def _norm(**kw):
    return _fill(fp4lin.fp4_qk_norm_args, dict(
        q_bf16=16, k_bf16=16, q_out_bf16=16, k_out_bf16=16, q_token_stride=256, q_head_stride=64, k_token_stride=128,
        k_head_stride=64, q_out_token_stride=256, q_out_head_stride=64, k_out_token_stride=128, k_out_head_stride=64,
        q_weight_bf16=16, k_weight_bf16=16, positions=16, tokens=3, q_heads=4, kv_heads=2, head_dim=64, eps=1e-6), kw)


def _rope_struct(**kw):
    return _fill(fp4lin.fp4_rope_params, dict(table=256, table_positions=8, rot_dim=64, layout=0, flags=0), kw)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), 2), (dict(q_heads=0), 2), (dict(kv_heads=-1), 2), (dict(head_dim=96), 2), (dict(head_dim=512), 2),
    (dict(tokens=1 << 30), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(q_bf16=None), 1), (dict(k_bf16=None), 1), (dict(q_out_bf16=None), 1), (dict(k_out_bf16=None), 1),
    (dict(q_weight_bf16=None), 1), (dict(k_weight_bf16=None), 1), (dict(positions=None), 1), (dict(positions=18), 3),
    (dict(q_bf16=24), 3), (dict(k_out_bf16=24), 3), (dict(q_weight_bf16=24), 3), (dict(k_weight_bf16=24), 3),
    (dict(q_token_stride=252), 3), (dict(k_out_head_stride=60), 3), (dict(q_head_stride=-64), 2)])
def test_norm_refusals(raw, kw, want):
    assert raw.fp4_qk_norm_rope(_norm(**kw), _rope_struct(), None) == want


def test_norm_more(raw):
    assert raw.fp4_qk_norm_rope(None, None, None) == 1
    assert raw.fp4_qk_norm_rope(_norm(tokens=0, q_bf16=None), _rope_struct(), None) == 0
    assert raw.fp4_qk_norm_rope(_norm(), _rope_struct(rot_dim=80), None) == 2
    assert raw.fp4_qk_norm_rope(_norm(), _rope_struct(layout=2), None) == 1


def _prompt(**kw):
    return _fill(fp4lin.fp4_prompt_attention_args, dict(
        q_bf16=16, k_bf16=16, v_bf16=16, out_bf16=16, lse=16, q_token_stride=256, q_head_stride=64, k_token_stride=128,
        k_head_stride=64, v_token_stride=128, v_head_stride=64, out_token_stride=256, out_head_stride=64, q_offsets=16,
        k_offsets=16, tokens=9, key_tokens=9, batch=2, q_heads=4, kv_heads=2, head_dim=64, causal=1, softmax_scale=0.125), kw)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 2), (dict(batch=65536), 2), (dict(tokens=-1), 2), (dict(tokens=1 << 31), 2), (dict(key_tokens=1 << 31), 2),
    (dict(key_tokens=-1), 2), (dict(q_heads=3), 2), (dict(q_heads=0), 2), (dict(kv_heads=0), 2), (dict(head_dim=96), 2),
    (dict(tokens=1 << 30, q_heads=8), 2), (dict(causal=2), 1), (dict(softmax_scale=0.0), 1),
    (dict(softmax_scale=float("inf")), 1), (dict(q_bf16=None), 1), (dict(k_bf16=None), 1), (dict(v_bf16=None), 1),
    (dict(out_bf16=None), 1), (dict(q_offsets=None), 1), (dict(k_offsets=None), 1), (dict(q_bf16=24), 3),
    (dict(k_bf16=24), 3), (dict(v_bf16=24), 3), (dict(out_bf16=24), 3), (dict(q_token_stride=252), 3),
    (dict(v_head_stride=60), 3), (dict(q_head_stride=-64), 2), (dict(k_token_stride=0), 2), (dict(v_head_stride=0), 2),
    (dict(k_token_stride=1 << 40), 2), (dict(lse=18), 3), (dict(q_offsets=18), 3), (dict(k_offsets=18), 3)])
def test_prompt_refusals(raw, kw, want):
    assert raw.fp4_prompt_attention(_prompt(**kw), 256, 1 << 40, None) == want


def test_prompt_more(raw):
    assert raw.fp4_prompt_attention(None, None, 0, None) == 1
    assert raw.fp4_prompt_attention(_prompt(tokens=0, q_bf16=None), None, 0, None) == 0
    size = raw.fp4_prompt_attention_workspace_size
    assert size(2, 9, 9, 4, 2, 96) == size(0, 9, 9, 4, 2, 64) == size(2, 0, 9, 4, 2, 64) == 0


def test_gemv_refusals(raw):
    ok = [16, 16, 16, None, 16, 2, 8, 64]

    def mx(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return raw.fp4_gemv_mxfp4(*a, None), raw.fp4_gemv_nvfp4(*a[:3], 1.0, *a[3:], None)

    assert mx(_5=9) == mx(_5=-1) == (2, 2)                      # rows
    assert mx(_6=0) == mx(_6=(1 << 24) + 1) == (2, 2)           # N
    assert mx(_7=48) == mx(_7=0) == mx(_7=65568) == (2, 2)      # K
    for i in (0, 1, 2, 4):
        assert mx(**{"_%d" % i: None}) == (1, 1)
        assert mx(**{"_%d" % i: 24}) == (3, 3)
    assert mx(_3=17) == (3, 3)
    assert mx(_5=0, _0=None) == (0, 0)

    def experts(x=16, ids=16, E=4, rows=2, per=1, w=16, sw=16, bias=None, out=16, N=8, K=64):
        return raw.fp4_gemv_mxfp4_experts(x, ids, E, rows, per, w, sw, bias, out, N, K, None)

    assert experts(E=0) == experts(E=1025) == experts(rows=-1) == experts(rows=65536) == experts(per=0) == 2
    assert experts(N=0) == experts(K=40) == 2
    assert experts(ids=None) == experts(x=None) == 1
    assert experts(ids=18) == experts(out=24) == 3
    assert experts(rows=0, x=None) == 0


def test_moe_refusals(raw):
    def dispatch(x=16, ids=16, tokens=3, top=2, E=4, width=64, xt=64, to=16, offsets=16, rows=16):
        return raw.fp4_moe_dispatch(x, ids, tokens, top, E, width, xt, to, offsets, rows, None)

    assert dispatch(tokens=-1) == dispatch(top=0) == dispatch(top=65) == dispatch(tokens=1 << 30, top=4) == 2
    assert dispatch(E=0) == dispatch(E=1025) == dispatch(width=60) == dispatch(width=0) == dispatch(width=(1 << 20) + 8) == 2
    assert dispatch(xt=-8) == 2
    assert dispatch(x=None) == dispatch(ids=None) == dispatch(to=None) == dispatch(offsets=None) == dispatch(rows=None) == 1
    assert dispatch(tokens=0, offsets=None) == 1
    assert dispatch(x=24) == dispatch(to=24) == dispatch(ids=18) == dispatch(offsets=18) == dispatch(rows=18) == dispatch(xt=60) == 3

    def combine(y=16, row_of=16, w=16, tokens=3, top=2, rows=6, width=64, out=16, ot=64):
        return raw.fp4_moe_combine(y, row_of, w, tokens, top, rows, width, out, ot, None)

    assert combine(rows=-1) == combine(top=0) == combine(width=4) == combine(tokens=-1) == 2
    assert combine(y=None) == combine(out=None) == 1
    assert combine(y=24) == combine(out=24) == combine(row_of=18) == combine(w=18) == combine(ot=4) == 3
    assert combine(tokens=0, y=None, out=None) == 0

    def backward(g=16, y=16, row_of=16, w=16, tokens=3, top=2, rows=6, width=64, gt=64, gy=16, gw=16):
        return raw.fp4_moe_combine_backward(g, y, row_of, w, tokens, top, rows, width, gt, gy, gw, None)

    assert backward(rows=-1) == backward(top=0) == backward(width=4) == backward(gt=-8) == 2
    assert backward(g=None) == backward(y=None) == backward(gy=None) == 1
    assert backward(g=24) == backward(y=24) == backward(gy=24) == backward(gw=18) == backward(gt=4) == 3
    assert backward(tokens=0, g=None) == 0


# -------------------------------------------------------------- the binding


def test_norm_binding(L):
    q, k, w, pos = _z(3, 4, 64), _z(3, 2, 64), _z(64), _z(3, dtype=I32)
    r = _rope(L)

    def call(q=q, k=k, qo=q, ko=k, qw=w, kw=w, pos=pos, rope=r):
        L.fp4_qk_norm_rope(q, k, qo, ko, qw, kw, 1e-6, pos, rope)

    for bad in (dict(qo=_z(3, 4, 32)), dict(ko=_z(2, 2, 64)), dict(k=_z(4, 2, 64), ko=_z(4, 2, 64)),
                dict(k=_z(3, 2, 128), ko=_z(3, 2, 128)), dict(qw=_z(32)), dict(kw=_z(64, dtype=F32)), dict(kw=_host(64)),
                dict(pos=_z(2, dtype=I32)), dict(pos=_z(3, dtype=I64)), dict(q=_host(3, 4, 64)),
                dict(q=_z(3, 4, 64, dtype=F32))):
        _refused(L, call, **bad)
    call()
    call(k=None, ko=None, kw=None)
    call(rope=None, pos=None)
    assert L._calls == ["fp4_qk_norm_rope"] * 3


def test_prompt_binding(L):
    q, k, cu = _z(9, 4, 64), _z(9, 2, 64), _z(3, dtype=I32)

    def call(q=q, k=k, v=k, out=q, cu=cu, cu_k=None, **kw):
        L.fp4_prompt_attention(q, k, v, out, cu, cu_k, **kw)

    for bad in (dict(out=_z(8, 4, 64)), dict(v=_z(9, 2, 128)), dict(k=_z(9, 2, 128), v=_z(9, 2, 128)), dict(cu=_z(3, dtype=I64)),
                dict(cu=_z(1, dtype=I32)), dict(cu_k=_z(2, dtype=I32)), dict(cu_k=_host(3, dtype=I32)),
                dict(lse=_z(8, 4, dtype=F32)), dict(lse=_z(9, 4)), dict(workspace=_host(8, dtype=U8)),
                dict(q=_z(9, 4, 64, dtype=F32)), dict(q=_z(9, 4, 128)[..., ::2])):
        _refused(L, call, **bad)
    call()
    call(cu_k=cu, lse=_z(9, 4, dtype=F32), workspace=_z(8, dtype=U8), causal=False)
    assert L._calls == ["fp4_prompt_attention"] * 2


def test_gemv_binding(L):
    x, w, s, out = _z(2, 128), _z(8, 64, dtype=U8), _z(512, dtype=U8), _z(2, 8)

    def call(x=x, w=w, s=s, b=None, out=out):
        L.fp4_gemv_mxfp4(x, w, s, b, out, 2, 8, 128)

    for bad in (dict(x=_z(128)), dict(x=_z(2, 128, dtype=F32)), dict(x=_z(2, 256)[:, ::2]), dict(w=_z(7, 64, dtype=U8)),
                dict(w=_z(8, 64)), dict(s=_z(511, dtype=U8)), dict(s=_host(512, dtype=U8)), dict(b=_z(7)),
                dict(b=_z(8, dtype=F32)), dict(out=_z(15)), dict(out=_host(2, 8))):
        _refused(L, call, **bad)
    _refused(L, L.fp4_gemv_nvfp4, x, w, s, 1.0, None, out, 2, 8, 128)   # twice the scales
    call(b=_z(8))
    L.fp4_gemv_nvfp4(x, w, _z(1024, dtype=U8), 1.0, None, out, 2, 8, 128)
    ids = _z(4, dtype=I32)
    we, se, oe = _z(3, 8, 64, dtype=U8), _z(3 * 512, dtype=U8), _z(4, 8)
    for bad in (dict(x=_z(128)), dict(w=w), dict(s=_z(2 * 512, dtype=U8)), dict(ids=_z(3, dtype=I32)),
                dict(ids=_z(4, dtype=I64)), dict(b=_z(23)), dict(out=_z(31))):
        a = dict(x=x, ids=ids, w=we, s=se, b=None, out=oe) | bad
        with pytest.raises(ValueError):
            L.fp4_gemv_mxfp4_experts(a["x"], a["ids"], 3, 4, 2, a["w"], a["s"], a["b"], a["out"], 8, 128)
    L.fp4_gemv_mxfp4_experts(x, ids, 3, 4, 2, we, se, _z(3, 8), oe, 8, 128)
    assert L._calls == ["fp4_gemv_mxfp4", "fp4_gemv_nvfp4", "fp4_gemv_mxfp4_experts"]


def test_moe_binding(L):
    x, ids, to, off, rows = _z(3, 64), _z(3, 2, dtype=I32), _z(6, 64), _z(5, dtype=I32), _z(3, 2, dtype=I32)

    def dispatch(x=x, ids=ids, to=to, off=off, rows=rows):
        L.fp4_moe_dispatch(x, ids, 4, to, off, rows)

    for bad in (dict(x=_z(4, 64)), dict(x=_z(3, 64, dtype=F32)), dict(x=_z(64, 3).t()), dict(ids=_z(6, dtype=I32)),
                dict(ids=_z(3, 2, dtype=I64)), dict(to=_z(5, 64)), dict(to=_z(6, 72)), dict(to=_z(6, 128)[:, :64]),
                dict(off=_z(4, dtype=I32)), dict(rows=_z(3, 1, dtype=I32)), dict(rows=_host(3, 2, dtype=I32))):
        _refused(L, dispatch, **bad)
    dispatch()
    w = _z(3, 2, dtype=F32)

    def combine(y=to, rows=rows, w=w, out=x, **kw):
        L.fp4_moe_combine(y, rows, w, out, **kw)

    for bad in (dict(y=_z(6, 128)[:, :64]), dict(out=_z(3, 72)), dict(out=_z(4, 64)), dict(w=_z(2, 2, dtype=F32)),
                dict(w=_z(3, 2)), dict(rows=_z(3, 2, dtype=I64)), dict(rows=None, w=None), dict(w=_z(3, 3, dtype=F32)),
                dict(rows=_z(2, 3, dtype=I32)), dict(rows=_z(6, dtype=I32)), dict(top_k=3)):
        _refused_more(L, combine, 1, **bad)
    combine()
    combine(rows=None)
    combine(rows=None, w=None, top_k=2)

    def backward(g=x, y=to, rows=rows, w=w, gy=to, gw=w):
        L.fp4_moe_combine_backward(g, y, rows, w, gy, gw)

    for bad in (dict(g=_z(4, 64)), dict(g=_z(3, 72)), dict(y=_z(5, 64)), dict(gy=_z(6, 64, dtype=F32)),
                dict(gw=_z(3, 1, dtype=F32)), dict(gw=_z(3, 3, dtype=F32)), dict(gy=_z(6, 128)[:, :64])):
        _refused_more(L, backward, 4, **bad)
    backward()
    backward(y=None, gw=None)
    assert L._calls == ["fp4_moe_dispatch"] + ["fp4_moe_combine"] * 3 + ["fp4_moe_combine_backward"] * 2


def _refused_more(L, call, before, **kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert len(L._calls) == before


def test_packed_arguments(L):
    """What the binding packs is the structures of the header, field by field."""
    v = tuple(range(1 << 40, (1 << 40) + 16)) + (5, 6, 7, 0.375)
    assert L._norm_args(*v) == bytes(L.fp4_qk_norm_args(*v))
    v = tuple(range(1 << 40, (1 << 40) + 17)) + (2, 3, 4, 5, 1, 0.375)
    assert L._prompt_args(*v) == bytes(L.fp4_prompt_attention_args(*v))
