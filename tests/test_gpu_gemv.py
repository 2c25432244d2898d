"""Matrix-vector products with 4-bit weights against the formula in 64 bits, on the
weights' exact values.

Bound.  Products are exact; the float32 sum of K of them is made of partial sums,
each addition off by at most 2^-23 of the magnitudes added so far (a tensor core's
additions may truncate), with K / 16 additions in a row at most; NVFP4's global
scale, the bias and the output's bf16 rounding follow:
  |out - ref| <= 2^-8 |ref| + (K / 16 + 40) 2^-23 (sum |x W| + |bias|)
and activations far below the largest of their block of 32 may be off by 2^-39 of
that."""
import numpy as np
import pytest

import _layer_ref as R
from _util import dev, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def swizzle(s):
    n, kb = s.shape
    p = np.zeros((-(-n // 128) * 128, -(-kb // 4) * 4), np.uint8)
    p[:n, :kb] = s
    return np.ascontiguousarray(p.reshape(-1, 4, 32, p.shape[1] // 4, 4).transpose(0, 3, 2, 1, 4)).reshape(-1)


def weight(r, n, k, nv, lo=None, hi=None):
    """codes [n, k / 2], scale bytes [n, k / group], the values in 64 bits."""
    c = r.integers(0, 16, (n, k)).astype(np.uint8)
    g = 16 if nv else 32
    lo, hi = (8, 0x7F) if nv and lo is None else (100, 140) if lo is None else (lo, hi)
    s = r.integers(lo, hi, (n, k // g)).astype(np.uint8)
    if nv:
        sv = R.element_values(s, R.MXFP8)
    else:
        sv = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return c[:, 0::2] | (c[:, 1::2] << 4), s, R.element_values(c, R.MXFP4) * sv.repeat(g, 1)


def acts(r, m, k):
    import torch

    x = r.standard_normal((m, k)) * np.where(r.random((m, k)) < 0.02, 100.0, 1.0) * 2.0 ** r.integers(-6, 7, (m, k))
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def check(out, x, w, bias, scale=1.0):
    x, out = x.double().numpy(), out.double().cpu().numpy()
    b = np.zeros(w.shape[0]) if bias is None else bias.double().numpy()
    k = w.shape[1]
    ref = (x @ w.T) * scale + b
    size = (np.abs(x) @ np.abs(w).T) * abs(scale) + np.abs(b)
    low = (np.abs(x).reshape(len(x), -1, 32).max(-1).repeat(32, 1) @ np.abs(w).T) * abs(scale) * 2.0 ** -39
    bound = 2.0 ** -8 * np.abs(ref) + (k / 16 + 40) * 2.0 ** -23 * size + low + 2.0 ** -126
    err = np.abs(out - ref)
    assert np.isfinite(out).all()
    assert (err <= bound).all(), float((err / bound).max())


CASES = [(1, 1, 32), (1, 8, 64), (2, 129, 96), (3, 130, 160), (4, 127, 512), (8, 300, 1024), (5, 64, 4128), (7, 33, 2080),
         (6, 257, 224), (8, 40, 16384), (8, 130, 12800), (2, 96, 65536), (8, 31, 65536), (1, 4096, 4096), (3, 1000, 7168)]


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("m,n,k", CASES)
def test_products(L, m, n, k, nv):
    import torch

    r = np.random.default_rng(m * n + k)
    codes, s, w = weight(r, n, k, nv)
    x = acts(r, m, k)
    bias = torch.from_numpy(r.standard_normal(n).astype(np.float32)).bfloat16() if n % 2 else None
    out = torch.full((m + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    b = None if bias is None else bias.cuda()
    if nv:
        L.fp4_gemv_nvfp4(x.cuda(), dev(codes), dev(swizzle(s)), -0.37, b, out[:m], m, n, k)
    else:
        L.fp4_gemv_mxfp4(x.cuda(), dev(codes), dev(swizzle(s)), b, out[:m], m, n, k)
    torch.cuda.synchronize()
    check(out[:m], x, w, bias, float(np.float32(-0.37)) if nv else 1.0)
    assert (out[m] == 7.0).all()


def test_extreme_scales(L):
    """E8M0 scales over their whole range in one row, subnormal 2^-127 among them, and
    activations that bring the products back."""
    import torch

    r = np.random.default_rng(1)
    n, k, m = 64, 512, 2
    codes, s, w = weight(r, n, k, False)
    s[:] = np.array([0, 1, 60, 120, 127, 128, 180, 200] * 2, np.uint8)
    w = R.element_values(np.stack((codes & 15, codes >> 4), -1).reshape(n, k), R.MXFP4) * (2.0 ** (s.astype(np.float64) - 127)).repeat(32, 1)
    back = 2.0 ** -(s[0].astype(np.float64) - 127).repeat(32)
    x = torch.from_numpy((r.standard_normal((m, k)) * np.clip(back, 2.0 ** -100, 2.0 ** 115)).astype(np.float32)).bfloat16()
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    L.fp4_gemv_mxfp4(x.cuda(), dev(codes), dev(swizzle(s)), None, out, m, n, k)
    check(out, x, w, None)


@pytest.mark.parametrize("nv", [False, True])
def test_wide_activations(L, nv):
    """A block's activations over 60 binades: the largest ones decide."""
    import torch

    r = np.random.default_rng(2)
    n, k, m = 96, 256, 3
    codes, s, w = weight(r, n, k, nv)
    x = torch.from_numpy((r.standard_normal((m, k)) * 2.0 ** r.integers(-60, 1, (m, k)) * 2.0 ** 20).astype(np.float32)).bfloat16()
    x[1] = 0.0
    x[2, 32:] = 0.0
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    args = (x.cuda(), dev(codes), dev(swizzle(s)))
    if nv:
        L.fp4_gemv_nvfp4(*args, 1.0, None, out, m, n, k)
    else:
        L.fp4_gemv_mxfp4(*args, None, out, m, n, k)
    check(out, x, w, None)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("nv", [False, True])
def test_nan_and_inf(L, nv):
    import torch

    r = np.random.default_rng(3)
    n, k, m = 70, 256, 3
    codes, s, w = weight(r, n, k, nv)
    s[5, 3] = 0x7F if nv else 0xFF                 # a NaN scale: row 5 of the weight
    x = acts(r, m, k)
    x[1, 100] = float("nan")                       # row 1 of the activations
    x[2, 40] = float("inf")
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    args = (x.cuda(), dev(codes), dev(swizzle(s)))
    if nv:
        L.fp4_gemv_nvfp4(*args, 1.0, None, out, m, n, k)
    else:
        L.fp4_gemv_mxfp4(*args, None, out, m, n, k)
    o = out.double().cpu().numpy()
    keep = np.arange(n) != 5
    assert np.isnan(o[:, 5]).all() and np.isnan(o[1]).all()
    check(out[:1][:, torch.from_numpy(keep).cuda()].contiguous(), x[:1], w[keep], None)
    at = w[keep, 40]
    want = np.where(at == 0, np.nan, np.where(at > 0, np.inf, -np.inf))
    assert np.array_equal(o[2, keep], want, equal_nan=True)


@pytest.mark.parametrize("tokens,top,E,n,k", [(1, 8, 64, 200, 512), (3, 2, 5, 130, 1024), (4, 4, 4, 37, 96), (1, 1, 1, 8, 32),
                                              (70, 3, 7, 40, 64)])
def test_experts(L, tokens, top, E, n, k):
    import torch

    r = np.random.default_rng(tokens + n)
    parts = [weight(r, n, k, False) for _ in range(E)]
    w = torch.stack([dev(c) for c, _, _ in parts])
    sw = torch.stack([dev(swizzle(s)) for _, s, _ in parts])
    bias = torch.from_numpy(r.standard_normal((E, n)).astype(np.float32)).bfloat16()
    ids = r.integers(0, E, (tokens, top)).astype(np.int32)
    if tokens > 1:
        ids[0, 0], ids[1, -1] = -1, E
    for per, rows_x in ((top, tokens), (1, tokens * top)):
        x = acts(r, rows_x, k)
        out = torch.full((tokens * top, n), 7.0, dtype=torch.bfloat16, device="cuda")
        L.fp4_gemv_mxfp4_experts(x.cuda(), dev(ids), E, tokens * top, per, w, sw, bias.cuda(), out, n, k)
        for i, e in enumerate(ids.reshape(-1)):
            if 0 <= e < E:
                check(out[i:i + 1], x[i // per:i // per + 1], parts[e][2], bias[e])
            else:
                assert (out[i] == 0).all()


def test_same_result_on_a_side_stream_and_in_a_graph(L):
    import torch

    r = np.random.default_rng(5)
    m, n, k = 4, 513, 1056
    codes, s, w = weight(r, n, k, False)
    x, c, sw = acts(r, m, k).cuda(), dev(codes), dev(swizzle(s))
    a, b, g = (torch.zeros(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    L.fp4_gemv_mxfp4(x, c, sw, None, a, m, n, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.fp4_gemv_mxfp4(x, c, sw, None, b, m, n, k)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.fp4_gemv_mxfp4(x, c, sw, None, g, m, n, k)
    graph.replay()
    torch.cuda.synchronize()
    check(a, x.cpu(), w, None)
    assert torch.equal(a, b) and torch.equal(a, g)


def test_calls_one_behind_the_other(L):
    """Thousands of calls that nothing waits between, on inputs in turns: the same bits
    every time (a ring whose places changed hands failed after about a thousand)."""
    import torch

    r = np.random.default_rng(6)
    for m, n, k in ((8, 2048, 7168), (1, 2048, 4096), (3, 1024, 4128)):
        sides = []
        for _ in range(3):
            codes, s, w = weight(r, n, k, False)
            x = acts(r, m, k)
            out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
            args = (x.cuda(), dev(codes), dev(swizzle(s)), None, out, m, n, k)
            L.fp4_gemv_mxfp4(*args)
            check(out, x, w, None)
            sides.append((args, out, out.clone()))
        for i in range(3000):
            L.fp4_gemv_mxfp4(*sides[i % 3][0])
        torch.cuda.synchronize()
        for _, out, first in sides:
            assert torch.equal(out, first)
        assert L.fp4_get_device_status() == 0
