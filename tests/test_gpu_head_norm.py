"""Norms of queries and keys with the rotation, against the formula in 64 bits.

Bound.  The sum of D squares is off by (16 + log2 D) 2^-24 of itself, and the mean,
square root, division, weight, and rotation add a rounding each: a normed element is
off by 24 2^-24 of itself, a turned one by that of both its terms, and then comes the
bf16 rounding: |out - ref| <= 2^-8 |ref| + 28 2^-24 (|a c| + |b s|)."""
import numpy as np
import pytest

import _layer_ref as R
from _util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def reference(x, w, eps, positions, table, rot, layout, inverse):
    """(values, sum of the terms' magnitudes)"""
    x, w = x.double().cpu().numpy(), w.double().cpu().numpy()
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * w
    if rot == 0:
        return y, np.abs(y)
    half = rot // 2
    t = table.double().cpu().numpy()[np.clip(positions.cpu().numpy(), 0, len(table) - 1)][:, None]
    c, s = t[..., :half], t[..., half:] * (-1 if inverse else 1)
    i = np.arange(half)
    a, b = (i, i + half) if layout == 0 else (2 * i, 2 * i + 1)
    out, size = y.copy(), np.abs(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
    size[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return out, size


def close(got, ref, size):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    bound = 2.0 ** -8 * np.abs(ref) + 28 * 2.0 ** -24 * size + 2.0 ** -133
    assert (np.abs(got - ref)[ok] <= bound[ok]).all()


def make(r, *shape):
    import torch

    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).bfloat16().cuda()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("t,hq,hkv,dim,rot", [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (7, 5, 1, 128, 64), (33, 3, 2, 256, 96),
                                              (64, 6, 0, 64, 16), (300, 7, 3, 128, 112), (5, 2, 2, 256, 256), (9, 4, 4, 128, 0)])
def test_norms(L, t, hq, hkv, dim, rot, layout, inverse):
    import torch

    r = np.random.default_rng(t * hq + dim + rot)
    qkv = make(r, t, (hq + 2 * hkv) * dim + 8)
    qkv *= torch.from_numpy(2.0 ** r.integers(-20, 20, (t, 1))).to(qkv)
    qkv[0, :dim] = 0.0   # a head of zeros
    q = qkv[:, : hq * dim].unflatten(1, (hq, dim))
    k = qkv[:, hq * dim: (hq + hkv) * dim].unflatten(1, (hkv, dim)) if hkv else None
    if t > 4 and k is not None:
        k[3, 0, 5] = float("nan")
        q[4, 0, 5] = float("inf")
    qw, kw = make(r, dim), make(r, dim)
    table = torch.from_numpy(r.standard_normal((50, max(rot, 16))).astype(np.float32)).cuda()
    pos = torch.from_numpy(r.integers(-3, 55, t).astype(np.int32)).cuda()
    rope = L.rope_params(table, rot, layout, inverse) if rot else None
    # one output with its heads outermost
    qo = torch.full((hq, t, dim), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ko = torch.full((t, hkv, dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")[..., :dim] if hkv else None
    before = qkv.clone()
    L.fp4_qk_norm_rope(q, k, qo, ko, qw, kw, 1e-6, pos, rope)
    assert torch.equal(qkv.view(torch.int16), before.view(torch.int16))
    with np.errstate(invalid="ignore"):
        close(qo, *reference(q, qw, 1e-6, pos, table, rot, layout, inverse))
        if hkv:
            close(ko, *reference(k, kw, 1e-6, pos, table, rot, layout, inverse))
    # in place: the same bits
    L.fp4_qk_norm_rope(q, k, q, k, qw, kw, 1e-6, pos, rope)
    assert torch.equal(q.contiguous().view(torch.int16), qo.contiguous().view(torch.int16))
    if hkv:
        assert torch.equal(k.contiguous().view(torch.int16), ko.contiguous().view(torch.int16))
    assert torch.equal(qkv[:, (hq + hkv) * dim:].contiguous().view(torch.int16), before[:, (hq + hkv) * dim:].contiguous().view(torch.int16))


def test_large_eps(L):
    import torch

    r = np.random.default_rng(0)
    q, w = make(r, 3, 2, 64), make(r, 64)
    out = torch.empty_like(q)
    L.fp4_qk_norm_rope(q, None, out, None, w, None, 3.5)
    close(out, *reference(q, w, 3.5, None, None, 0, 0, False))
