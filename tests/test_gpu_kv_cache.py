"""Rotary positions and the MX-quantized paged cache on the GPU against their
formulas.

rope: |out - ref| <= 2^-8 |ref| (the bf16 rounding, 1 % more for what is
rounded) + 3 float32 roundings of the two products: 2^-23 (|a c| + |b s|).
append: codes and scales bit for bit those of float32 with one operation at a
time.  read: the exact value, rounded once to bf16."""
import numpy as np
import pytest

import _layer_ref as R
from _util import bf16_bits_host, bf16_bits_to_f64, dev, dev_bf16, host, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def _bits(r, shape, scale=1.0):
    import torch

    x = torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).bfloat16()
    return x.view(torch.int16).numpy().view(np.uint16)


def _table(positions, rot, base=10000.0):
    a = np.arange(positions)[:, None] * R.rope_frequencies(rot, base)
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def _f32(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_table(L, kind, rot):
    import torch

    P = 5000
    t = torch.empty(P, rot, device="cuda")
    kw = dict(factor=8.0, original_positions=1024, turns_fast=32.0, turns_slow=1.0, magnitude=1.25) if kind == 2 else \
        dict(factor=4.0)
    L.fp4_rope_table(t, P, rot, 10000.0, kind, **kw)
    w = R.rope_frequencies(rot, 10000.0, kind, kw["factor"], kw.get("original_positions", 0))
    a = np.arange(P)[:, None] * w
    mag = kw.get("magnitude", 1.0)
    want = np.concatenate((np.cos(a), np.sin(a)), 1) * mag
    # one float32 rounding; the angle (up to 5000) carries a few 64-bit roundings
    assert np.max(np.abs(host(t) - want)) <= 2.0 ** -24 * mag + 1e-11


@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (7, 3, 128, 128), (33, 5, 128, 64), (5, 2, 64, 48), (3, 2, 192, 96),
                                       (257, 8, 128, 16)])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("gap", [0, 8])
def test_rope(L, T, H, D, rot, layout, gap):
    import torch

    r = np.random.default_rng(T + rot)
    bits = _bits(r, (T, H * (D + gap) + 2 * gap))
    P = 300
    table, pos = _table(P, rot), r.integers(-3, P + 5, T).astype(np.int32)
    x = dev_bf16(bits)[:, gap:gap + H * (D + gap)].unflatten(1, (H, D + gap))[:, :, :D]
    xf = _f32(bits)[:, gap:gap + H * (D + gap)].reshape(T, H, D + gap)[:, :, :D]
    rope = L.rope_params(dev(table), rot, layout)
    out = torch.full((T, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.fp4_rope(x, out, dev(pos), rope)
    cs = table[np.clip(pos, 0, P - 1)].astype(np.float64)
    ref = R.rotate(xf, cs[:, :rot // 2], cs[:, rot // 2:], rot, layout)
    mag = R.rotate(np.abs(xf), np.abs(cs[:, :rot // 2]), -np.abs(cs[:, rot // 2:]), rot, layout)
    mag = np.maximum(np.abs(mag), np.abs(R.rotate(np.abs(xf), np.abs(cs[:, :rot // 2]), np.abs(cs[:, rot // 2:]), rot, layout)))
    got = bf16_bits_to_f64(bf16_bits_host(out))
    assert np.all(np.abs(got - ref) <= 1.01 * 2.0 ** -8 * np.abs(ref) + 2.0 ** -23 * mag + 1e-38)
    # bit for bit the float32 operations, one at a time
    f = R.rotate(xf, table[np.clip(pos, 0, P - 1)][:, :rot // 2], table[np.clip(pos, 0, P - 1)][:, rot // 2:], rot, layout,
                 np.float32)
    assert np.array_equal(bf16_bits_host(out), bf16_bits_host(torch.from_numpy(f).bfloat16()))
    # in place, and the inverse undoes it up to two bf16 roundings
    L.fp4_rope(x, x, dev(pos), rope)
    assert torch.equal(x, out)
    L.fp4_rope(out, out, dev(pos), L.rope_params(dev(table), rot, layout, inverse=True))
    back = bf16_bits_to_f64(bf16_bits_host(out))
    # the first call's rounding of both elements of a pair, turned back, and the second's own
    pair = np.abs(got)
    i, j = R.pairs(rot, layout)
    c, s = np.abs(cs[:, None, :rot // 2]), np.abs(cs[:, None, rot // 2:])
    first = pair.copy()
    first[..., i], first[..., j] = pair[..., i] * c + pair[..., j] * s, pair[..., j] * c + pair[..., i] * s
    assert np.all(np.abs(back - xf) <= 1.01 * 2.0 ** -8 * (first + np.abs(xf)) + 2.0 ** -21 * first + 1e-38)


def test_rope_gradient_is_the_inverse_rotation(L):
    """<dy, rope(x)> changes by <rope^-1(dy), dx>: the inverse is the transposed
    map, against the formula's gradient and against differences of it."""
    import torch

    r = np.random.default_rng(4)
    T, H, D, rot = 6, 2, 64, 32
    table, pos = _table(50, rot), np.arange(T, dtype=np.int32) * 7
    dy = _bits(r, (T, H, D))
    for layout in (0, 1):
        dx = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
        L.fp4_rope(dev_bf16(dy), dx, dev(pos), L.rope_params(dev(table), rot, layout, inverse=True))
        c, s = table[pos][:, :rot // 2].astype(np.float64), table[pos][:, rot // 2:].astype(np.float64)
        g = bf16_bits_to_f64(dy)
        got = bf16_bits_to_f64(bf16_bits_host(dx))
        x = r.standard_normal((T, H, D))
        for t, h, d in r.integers(0, (T, H, D), (40, 3)):
            e = np.zeros_like(x)
            e[t, h, d] = 0.5
            diff = (g * (R.rotate(x + e, c, s, rot, layout) - R.rotate(x - e, c, s, rot, layout))).sum()
            assert abs(diff - got[t, h, d]) <= 2.0 ** -8 * (np.abs(g[t, h]).max() + abs(diff)) + 1e-12


def _cache(L, fmt, pages, heads, page, dim, fill=0xA5):
    import torch

    width = dim if fmt == R.MXFP8 else dim // 2
    t = [torch.full((pages, heads, page, w), fill, dtype=torch.uint8, device="cuda") for w in (width, dim // 32) * 2]
    return L.kv_cache(*t, page, fmt)


CACHES = [(1, 1, 16, 64), (9, 2, 16, 128), (40, 8, 48, 128), (130, 3, 64, 64)]


@pytest.mark.parametrize("T,heads,page,dim", CACHES)
@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("rope", [None, (0, 1), (0, 2), (1, 1), (1, 2)])
def test_append_is_exact(L, T, heads, page, dim, fmt, rope):
    r = np.random.default_rng(T + dim)
    gap = 8 * heads
    kv = _bits(r, (T, 2 * heads * dim + gap), 3.0)
    kv[0, :32] = 0
    kv[T // 2, 3] = 0x7FC0
    kv[T - 1, heads * dim + 5] = 0xFF80
    k, v = kv[:, :heads * dim].reshape(T, heads, dim), kv[:, heads * dim:2 * heads * dim].reshape(T, heads, dim)
    kvd = dev_bf16(kv)
    kd, vd = kvd[:, :heads * dim].unflatten(1, (heads, dim)), kvd[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
    pages = -(-2 * T // page) + 1
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[3], slots[4] = -1, pages * page       # padding: skipped
    cache = _cache(L, fmt, pages, heads, page, dim)
    kf, vf = _f32(k), _f32(v)
    args = {}
    if rope:
        layout, part = rope
        rot = dim // part
        table, pos = _table(100, rot), r.integers(0, 100, T).astype(np.int32)
        args = dict(rope=L.rope_params(dev(table), rot, layout), positions=dev(pos))
        with np.errstate(invalid="ignore"):
            kf = R.rotate(kf, table[pos][:, :rot // 2], table[pos][:, rot // 2:], rot, layout, np.float32)
    L.fp4_kv_append(cache, kd, vd, dev(slots), **args)
    for x, codes_t, scales_t in ((kf, *cache.tensors[:2]), (vf, *cache.tensors[2:])):
        codes, scales = R.mx_quantize(x, fmt)
        wc = np.full(codes_t.shape, 0xA5, np.uint8)
        ws = np.full(scales_t.shape, 0xA5, np.uint8)
        for t in range(T):
            if 0 <= slots[t] < pages * page:
                wc[slots[t] // page, :, slots[t] % page] = R.pack(codes[t], fmt)
                ws[slots[t] // page, :, slots[t] % page] = scales[t]
        assert np.array_equal(host(scales_t), ws)
        assert np.array_equal(host(codes_t), wc)


def test_append_without_rotation_matches_the_activation_quantizer(L):
    """The cache holds what the library's activation quantizers make of the rows."""
    import torch

    r = np.random.default_rng(0)
    T, dim = 48, 128
    k, v = _bits(r, (T, 1, dim)), _bits(r, (T, 1, dim))
    for fmt, call in ((R.MXFP8, "fp4_quant_act_mxfp8"), (R.MXFP4, "fp4_quant_act_mxfp4")):
        cache = _cache(L, fmt, 1, 1, T, dim)
        L.fp4_kv_append(cache, dev_bf16(k), dev_bf16(v), torch.arange(T, device="cuda"))
        for bits, codes, scales in ((k, *cache.tensors[:2]), (v, *cache.tensors[2:])):
            c, s = torch.empty_like(codes), torch.empty_like(scales)
            getattr(L, call)(dev_bf16(bits.reshape(T, dim)), c, s, T, dim, sf_layout=L.FP4_SF_ROWMAJOR)
            assert torch.equal(c, codes) and torch.equal(s, scales)


@pytest.mark.parametrize("lens,heads,page,dim", [([1], 1, 16, 64), ([5, 0, 33, 16], 2, 16, 128), ([100, 47], 8, 48, 128),
                                                 ([0, 0, 3], 3, 64, 64)])
@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_read_is_exact(L, lens, heads, page, dim, fmt):
    import torch

    r = np.random.default_rng(sum(lens) + dim)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 3
    order = r.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(max(per), 1) + 1), 2 ** 30, np.int32)       # unused entries are never followed
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    cache = _cache(L, fmt, pages, heads, page, dim)
    vals = []
    for codes_t, scales_t in (cache.tensors[:2], cache.tensors[2:]):
        c = r.integers(0, 256, tuple(codes_t.shape)).astype(np.uint8)
        if fmt == R.MXFP8:
            c[(c & 127) == 127] = 0x7E
        s = r.integers(90, 160, tuple(scales_t.shape)).astype(np.uint8)
        s[r.uniform(size=s.shape) < 0.01] = 255
        s[0, 0, 0, 0] = 0
        codes_t.copy_(dev(c))
        scales_t.copy_(dev(s))
        vals.append(R.mx_values(R.unpack(c, fmt), s, fmt))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    out = [torch.full((cu[-1], heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.fp4_kv_read(cache, dev(table), dev(cu), *out)
    for o, v in zip(out, vals):
        want = np.concatenate([v[table[b, t // page], :, t % page][None] for b, n in enumerate(lens) for t in range(n)])
        assert np.array_equal(bf16_bits_to_f64(bf16_bits_host(o)),
                              bf16_bits_to_f64(bf16_bits_host(torch.from_numpy(want).bfloat16())), equal_nan=True)


def test_read_skips_pages_outside_the_cache(L):
    import torch

    cache = _cache(L, R.MXFP8, 2, 1, 16, 64, fill=0x38)
    cache.tensors[1].fill_(127)
    cache.tensors[3].fill_(127)
    table = dev(np.array([[0, -1], [7, 1]], np.int32))
    cu = dev(np.array([0, 32, 80], np.int32))           # the second sequence is longer than its table row
    k, v = (torch.full((80, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.fp4_kv_read(cache, table, cu, k, v)
    want = [1.0] * 16 + [7.0] * 16 + [7.0] * 16 + [1.0] * 16 + [7.0] * 16
    assert k[:, 0, 0].tolist() == want and v[:, 0, 63].tolist() == want


def test_offsets_past_32_bits(L):
    """A cache of more than 4 GB per array: appended and read at its end."""
    import torch

    heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (heads * page * dim) + 4
    t = [torch.empty((pages, heads, page, w), dtype=torch.uint8, device="cuda") for w in (dim, dim // 32) * 2]
    cache = L.kv_cache(*t, page, R.MXFP8)
    r = np.random.default_rng(2)
    k, v = _bits(r, (3, heads, dim)), _bits(r, (3, heads, dim))
    slots = np.array([pages * page - 1, pages * page - 70, 5], np.int64)
    L.fp4_kv_append(cache, dev_bf16(k), dev_bf16(v), dev(slots))
    codes, scales = R.mx_quantize(_f32(k), R.MXFP8)
    for i, s in enumerate(slots):
        assert np.array_equal(host(t[0][s // page, :, s % page]), codes[i])
        assert np.array_equal(host(t[1][s // page, :, s % page]), scales[i])
    table = dev(np.array([[pages - 1]], np.int32))
    ko, vo = (torch.zeros((page, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.fp4_kv_read(cache, table, dev(np.array([0, page], np.int32)), ko, vo)
    want = R.mx_values(*R.mx_quantize(_f32(v), R.MXFP8), R.MXFP8)[0]
    assert np.array_equal(bf16_bits_to_f64(bf16_bits_host(vo[-1])), want)


def test_a_table_of_one_row_may_have_any_stride(L):
    import torch

    cache = _cache(L, R.MXFP8, 2, 1, 16, 64, fill=0x38)
    cache.tensors[1].fill_(127)
    cache.tensors[3].fill_(127)
    table = torch.tensor([1, 0], dtype=torch.int32, device="cuda").as_strided((1, 2), (0, 1))
    k, v = (torch.zeros((20, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.fp4_kv_read(cache, table, dev(np.array([0, 20], np.int32)), k, v)
    assert torch.all(k == 1.0) and torch.all(v == 1.0)
