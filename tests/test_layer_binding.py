"""The binding's checks of the layer operators' tensors: one that does not fit
would be read or written past its end, or as another type.  Every refusal is a
ValueError before the library is called.  No device is touched: the library is a
stand-in that counts its calls, the tensors are host tensors that say otherwise."""
import pytest
import torch

from nvfp4_mxfp4_w4a4_gb300 import attention_block
from nvfp4_mxfp4_w4a4_gb300 import fp4lin


class _Device(torch.Tensor):
    is_cuda = True


class _Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def L(monkeypatch):
    library = _Library()
    monkeypatch.setattr(fp4lin, "load", lambda: library)
    monkeypatch.setattr(fp4lin, "_stream", lambda s: 0)
    monkeypatch.setattr(fp4lin, "_calls", library.calls, raising=False)
    return fp4lin


def _refused(L, call, *args, **kw):
    with pytest.raises(ValueError):
        call(*args, **kw)
    assert not L._calls


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Device)


def _host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32, I64, F32, U8 = torch.int32, torch.int64, torch.float32, torch.uint8


def _cache(L, **kw):
    t = dict(k_codes=_z(4, 2, 16, 64, dtype=U8), k_scales=_z(4, 2, 16, 2, dtype=U8), v_codes=_z(4, 2, 16, 64, dtype=U8),
             v_scales=_z(4, 2, 16, 2, dtype=U8))
    t.update(kw)
    return L.kv_cache(*t.values(), 16, L.FP4_ACT_MXFP8)


def _rope(L):
    return L.rope_params(_z(8, 64, dtype=F32), 64)


@pytest.mark.parametrize("table,rot", [(_z(8, 64, dtype=torch.float64), 64), (_z(8, 64), 64), (_z(8, 64, dtype=F32), 128),
                                       (_z(8, 64, dtype=F32), 32), (_z(512, dtype=F32), 64),
                                       (_z(64, 8, dtype=F32).t(), 64), (_z(8, 128, dtype=F32)[:, :64], 64),
                                       (_host(8, 64, dtype=F32), 64)])
def test_rope_tables(L, table, rot):
    _refused(L, L.rope_params, table, rot)


@pytest.mark.parametrize("table", [_z(9, 64), _z(8, 64, dtype=F32), _z(64, 9, dtype=F32).t(), _host(9, 64, dtype=F32)])
def test_tables_to_fill(L, table):
    _refused(L, L.fp4_rope_table, table, 9, 64, 10000.0)
    L.fp4_rope_table(_z(9, 64, dtype=F32), 9, 64, 10000.0)
    assert L._calls == ["fp4_rope_table"]


@pytest.mark.parametrize("kw", [
    dict(k_codes=_z(4, 2, 16, 64, dtype=I32)), dict(v_scales=_z(4, 2, 16, 2, dtype=F32)),
    dict(v_codes=_z(4, 2, 16, 32, dtype=U8)), dict(k_codes=_z(4, 2, 16, 128, dtype=U8)[..., ::2]),
    dict(v_codes=_host(4, 2, 16, 64, dtype=U8))])
def test_caches(L, kw):
    _refused(L, _cache, L, **kw)
    assert _cache(L).struct.num_pages == 4


@pytest.mark.parametrize("kw", [
    dict(x=_z(5, 3, 64, dtype=F32)), dict(out=_z(5, 3, 64, dtype=torch.float16)), dict(out=_z(5, 3, 128)),
    dict(positions=_z(5, dtype=I64)), dict(positions=_z(4, dtype=I32)), dict(positions=_z(10, dtype=I32)[::2]),
    dict(x=_z(5, 64, 3).transpose(1, 2)), dict(x=_host(5, 3, 64)), dict(positions=_host(5, dtype=I32))])
def test_rope(L, kw):
    t = dict(x=_z(5, 3, 64), out=_z(5, 3, 64), positions=_z(5, dtype=I32))
    _refused(L, L.fp4_rope, *{**t, **kw}.values(), _rope(L))
    t["x"] = _z(5, 512)[:, 64:256].unflatten(1, (3, 64))
    L.fp4_rope(*t.values(), _rope(L))
    assert L._calls == ["fp4_rope"]


@pytest.mark.parametrize("kw", [
    dict(k=_z(5, 2, 64, dtype=F32)), dict(v=_z(5, 2, 64, dtype=F32)), dict(v=_z(4, 2, 64)), dict(k=_z(5, 4, 64), v=_z(5, 4, 64)),
    dict(slots=_z(5, dtype=I32)), dict(slots=_z(4, dtype=I64)), dict(slots=_z(10, dtype=I64)[::2]),
    dict(positions=_z(5, dtype=I64)), dict(positions=_z(4, dtype=I32)), dict(v=_host(5, 2, 64)), dict(slots=_host(5, dtype=I64))])
def test_append(L, kw):
    def call(k, v, slots, positions):
        L.fp4_kv_append(_cache(L), k, v, slots, rope=_rope(L), positions=positions)

    t = dict(k=_z(5, 2, 64), v=_z(5, 2, 64), slots=_z(5, dtype=I64), positions=_z(5, dtype=I32))
    _refused(L, call, **{**t, **kw})
    call(**t)
    L.fp4_kv_append(_cache(L), t["k"], t["v"], t["slots"])
    assert L._calls == ["fp4_kv_append"] * 2


@pytest.mark.parametrize("kw", [
    dict(table=_z(3, 4, dtype=I64)), dict(table=_z(12, dtype=I32)), dict(table=_z(4, 3, dtype=I32).t()),
    dict(cu=_z(4, dtype=I64)), dict(cu=_z(3, dtype=I32)), dict(cu=_z(8, dtype=I32)[::2]),
    dict(k=_z(7, 2, 64, dtype=F32)), dict(v=_z(7, 2, 64, dtype=F32)), dict(k=_z(7, 1, 64), v=_z(7, 1, 64)),
    dict(k=_z(7, 2, 32), v=_z(7, 2, 32)), dict(v=_z(7, 4, 64)[:, ::2]), dict(table=_host(3, 4, dtype=I32)),
    dict(k=_host(7, 2, 64))])
def test_read(L, kw):
    def call(table, cu, k, v):
        L.fp4_kv_read(_cache(L), table, cu, k, v)

    t = dict(table=_z(3, 4, dtype=I32), cu=_z(4, dtype=I32), k=_z(7, 2, 64), v=_z(7, 2, 64))
    _refused(L, call, **{**t, **kw})
    call(**t)
    call(**{**t, "table": _z(3, 9, dtype=I32)[:, :4]})
    assert L._calls == ["fp4_kv_read"] * 2


@pytest.mark.parametrize("kw", [
    dict(q=_z(5, 4, 64, dtype=F32)), dict(out=_z(5, 4, 64, dtype=F32)), dict(out=_z(4, 4, 64)), dict(table=_z(3, 4, dtype=I64)),
    dict(table=_z(4, 3, dtype=I32).t()), dict(ctx=_z(3, dtype=I64)), dict(ctx=_z(2, dtype=I32)), dict(cu=_z(4, dtype=I64)),
    dict(cu=_z(3, dtype=I32)), dict(mask=_z(5, 1, dtype=I64)), dict(mask=_z(4, 1, dtype=I32)), dict(mask=_z(5, dtype=I32)),
    dict(mask=_z(5, 2, dtype=I32)[:, :1]), dict(lse=_z(5, 4)), dict(lse=_z(4, 5, dtype=F32).t()),
    dict(lse=_z(4, 4, dtype=F32)), dict(ws=_z(64, dtype=U8)[::2]), dict(ws=_host(64, dtype=U8)), dict(q=_host(5, 4, 64)),
    dict(ctx=_host(3, dtype=I32)), dict(lse=_host(5, 4, dtype=F32))])
def test_attention(L, kw):
    def call(q, out, table, ctx, cu, mask, lse, ws):
        L.fp4_kv_attention(_cache(L), q, out, table, ctx, cu, 64, 8, ws, tree_mask=mask, lse=lse)

    t = dict(q=_z(5, 4, 64), out=_z(5, 4, 64), table=_z(3, 4, dtype=I32), ctx=_z(3, dtype=I32), cu=_z(4, dtype=I32),
             mask=None, lse=None, ws=None)
    _refused(L, call, **{**t, **kw})
    call(**t)
    for dtype in (I32, torch.uint32):
        call(**{**t, "mask": _z(5, 1, dtype=dtype), "lse": _z(5, 4, dtype=F32), "ws": _z(64, dtype=U8)})
    assert L._calls == ["fp4_kv_attention"] * 3


@pytest.mark.parametrize("kw", [
    dict(codes=_z(256, 128, dtype=I32)), dict(codes=_z(128, 256, dtype=U8).t()), dict(scales=_z(2, 1)),
    dict(scales=_z(1, 1, dtype=F32)), dict(scales=_z(2, 2, dtype=F32)), dict(bias=_z(256, dtype=F32)), dict(bias=_z(128)),
    dict(codes=_host(256, 128, dtype=U8)), dict(scales=_host(2, 1, dtype=F32))])
def test_fp8_layers(L, kw):
    t = dict(codes=_z(256, 128, dtype=U8), scales=_z(2, 1, dtype=F32), bias=_z(256))
    _refused(L, attention_block.Fp8Linear, **{**t, **kw})
    attention_block.Fp8Linear(**t)


@pytest.mark.parametrize("x,out", [
    (_z(4, 128, dtype=F32), _z(4, 256)), (_z(4, 256)[:, :128], _z(4, 256)), (_z(4, 64), _z(4, 256)), (_z(128, 4).t(), _z(4, 256)),
    (_z(4, 128), _z(4, 128)), (_z(4, 128), _z(3, 256)), (_z(4, 128), _z(4, 256, dtype=F32)), (_z(4, 128), _z(256, 4).t()),
    (_host(4, 128), _z(4, 256)), (_z(4, 128), _host(4, 256))])
def test_fp8_layer_inputs(L, x, out):
    layer = attention_block.Fp8Linear(_z(256, 128, dtype=U8), _z(2, 1, dtype=F32))
    _refused(L, layer, x, out, _z(1 << 16, dtype=U8))
    layer(_z(4, 128), _z(4, 256), _z(1 << 16, dtype=U8))
    assert L._calls == ["fp4_linear_fp8_b128"]


@pytest.mark.parametrize("w", [_z(256, 128, dtype=F32), _z(128, 256).t(), _host(256, 128)])
def test_fp8_layer_weights(L, w):
    _refused(L, attention_block.Fp8Linear.from_bf16, w)


def test_packed_attention_arguments(L):
    """What the binding packs is the structure of the header, field by field."""
    v = (1 << 40, 2 << 40, 3 << 40, 4, 5, 6, 7, 8 << 40, 9, 10 << 40, 11 << 40, 12 << 40, 13, 14, 15 << 33, 16, 17, 18 << 33, 0.375)
    assert L._attention_args(*v) == bytes(L.fp4_kv_attention_args(*v))
