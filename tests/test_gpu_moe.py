"""Tokens sorted by expert and back, with weights, and the gradient; and the run of
them around the grouped FP4 layer.

Bounds.  A sum of k float32 products is off by k 2^-23 of the magnitudes, a bf16
output by 2^-8 of itself.  The gradient of a weight is a float32 sum of `width`
exact products, width / 32 + 5 additions in a row: off by that many times 2^-24 of
the magnitudes, twice for the products' own roundings."""
import numpy as np
import pytest

from _util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def sort_rows(ids, E):
    """row_of and row_offsets by the definition."""
    row_of, offsets, at = np.full(ids.shape, -1, np.int32), [0], 0
    for e in range(E):
        for t, j in np.argwhere(ids == e):
            row_of[t, j] = at
            at += 1
        offsets.append(at)
    return row_of, np.array(offsets, np.int32)


CASES = [(1, 1, 1, 8), (1, 8, 64, 64), (5, 3, 2, 24), (32, 8, 64, 1032), (33, 2, 1024, 16), (127, 8, 16, 136), (129, 8, 7, 4096),
         (1000, 5, 40, 72), (4097, 8, 256, 8), (700, 64, 1000, 8), (513, 2, 1, 2048)]


def routing(r, tokens, top, E, kind):
    ids = r.integers(0, E, (tokens, top)).astype(np.int32)
    if kind == "padded":
        ids[r.random(tokens) < 0.3] = -1
        ids[r.random((tokens, top)) < 0.1] = E + 3
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "none":
        ids[:] = -5
    return ids


@pytest.mark.parametrize("kind", ["plain", "padded", "one", "none"])
@pytest.mark.parametrize("tokens,top,E,width", CASES)
def test_dispatch(L, tokens, top, E, width, kind):
    import torch

    r = np.random.default_rng(tokens + width)
    ids = routing(r, tokens, top, E, kind)
    x = torch.from_numpy(r.standard_normal((tokens, width + 16)).astype(np.float32)).bfloat16().cuda()[:, 8:8 + width]
    to = torch.full((tokens * top, width), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    rows = torch.full((tokens, top), -9, dtype=torch.int32, device="cuda")
    L.fp4_moe_dispatch(x, torch.from_numpy(ids).cuda(), E, to, off, rows)
    want_rows, want_off = sort_rows(ids, E) if tokens * E < 200000 else fast_rows(ids, E)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(rows.cpu().numpy(), want_rows)
    expect = torch.full((tokens * top, width), 7.0, dtype=torch.bfloat16)
    t, j = np.nonzero(want_rows >= 0)
    expect[torch.from_numpy(want_rows[t, j]).long()] = x.cpu()[torch.from_numpy(t)]
    assert torch.equal(to.cpu(), expect)


# Few pairs: whole blocks of one token, blocks of several, the last one short, 64 choices.
FEW = [(128, 8, 1024, 1032), (1024, 1, 64, 520), (16, 64, 100, 1024), (7, 16, 33, 256), (61, 4, 1, 72), (9, 3, 2, 1048), (1, 64, 1024, 2048),
       (63, 8, 33, 512), (61, 4, 1, 256), (64, 16, 9, 4104)]


@pytest.mark.parametrize("kind", ["plain", "padded", "one", "none"])
@pytest.mark.parametrize("tokens,top,E,width", FEW)
def test_dispatch_of_few(L, tokens, top, E, width, kind):
    test_dispatch(L, tokens, top, E, width, kind)


def fast_rows(ids, E):
    key = np.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    order = np.argsort(key, kind="stable")
    row = np.empty(key.size, np.int32)
    row[order] = np.arange(key.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]).astype(np.int32)
    return np.where(key < E, row, -1).reshape(ids.shape).astype(np.int32), offsets


def test_dispatch_of_many(L):
    """More pairs than one round of the sorting threads, offsets past 2^31 bytes."""
    import torch

    r = np.random.default_rng(0)
    tokens, top, E, width = 150001, 8, 200, 1032
    ids = routing(r, tokens, top, E, "padded")
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    to = torch.zeros(tokens * top, width, dtype=torch.bfloat16, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows = torch.empty(tokens, top, dtype=torch.int32, device="cuda")
    L.fp4_moe_dispatch(x, torch.from_numpy(ids).cuda(), E, to, off, rows)
    want_rows, want_off = fast_rows(ids, E)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(rows.cpu().numpy(), want_rows)
    t, j = np.nonzero(want_rows >= 0)
    for part in np.array_split(np.arange(t.size), 8):
        assert torch.equal(to[torch.from_numpy(want_rows[t[part], j[part]]).long().cuda()], x[torch.from_numpy(t[part]).cuda()])
    assert (to[int(want_off[-1]):] == 0).all()


def test_no_tokens(L):
    import torch

    off = torch.full((5,), -9, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    L.fp4_moe_dispatch(none, ids, 4, none, off, ids)
    assert (off == 0).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("identity", [False, True])
@pytest.mark.parametrize("tokens,top,E,width", CASES)
def test_combine_and_gradient(L, tokens, top, E, width, identity, weighted):
    import torch

    r = np.random.default_rng(tokens * 3 + width)
    if identity:
        row_of = np.arange(tokens * top, dtype=np.int32).reshape(tokens, top)
    else:
        row_of, _ = fast_rows(routing(r, tokens, top, E, "padded"), E)
    rows = tokens * top
    y = torch.from_numpy(r.standard_normal((rows, width)).astype(np.float32)).bfloat16()
    y[rows // 2, 0] = float("nan")
    w = r.random((tokens, top)).astype(np.float32)
    grad = torch.from_numpy(r.standard_normal((tokens, width + 8)).astype(np.float32)).bfloat16()[:, :width]
    out = torch.full((tokens, width + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    wd = torch.from_numpy(w).cuda() if weighted else None
    rd = None if identity else torch.from_numpy(row_of).cuda()
    L.fp4_moe_combine(y.cuda(), rd, wd, out[:, :width], top_k=top)
    gy = torch.full((rows, width), 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((tokens, top), 7.0, dtype=torch.float32, device="cuda")
    gd = torch.zeros(tokens, width + 8, dtype=torch.bfloat16, device="cuda")[:, :width].copy_(grad)
    L.fp4_moe_combine_backward(gd, y.cuda(), rd, wd, gy, gw, top_k=top)
    only = torch.full_like(gy, 7.0)
    L.fp4_moe_combine_backward(gd, None, rd, wd, only, top_k=top)
    yy, gg = y.double().numpy(), grad.double().numpy()
    ww = w.astype(np.float64) if weighted else np.ones((tokens, top))
    live = row_of >= 0
    got = yy[np.maximum(row_of, 0)]
    ref = np.where(live[..., None], ww[..., None] * got, 0.0).sum(1)
    size = np.where(live[..., None], ww[..., None] * np.abs(got), 0.0).sum(1)
    o = out.double().cpu().numpy()
    assert (o[:, width:] == 7.0).all()
    close(o[:, :width], ref, 2.0 ** -8 * np.abs(ref) + top * 2.0 ** -23 * size)
    ref = np.where(live, np.einsum("tjw,tw->tj", got, gg), 0.0)
    size = np.where(live, np.einsum("tjw,tw->tj", np.abs(got), np.abs(gg)), 0.0)
    close(gw.double().cpu().numpy(), ref, 2 * (width / 32 + 5) * 2.0 ** -24 * size)
    want = np.full((rows, width), 7.0)
    want[row_of[live]] = (ww[..., None] * gg[:, None])[live]
    close(gy.double().cpu().numpy(), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -149)
    assert torch.equal(gy, only)


def close(got, ref, bound):
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= bound[ok]).all(), float((np.abs(got - ref)[ok] / np.maximum(bound[ok], 1e-300)).max())


def test_gradient_by_differences(L):
    """The gradients against central differences of sum(grad * combine), whose map is
    linear in y and in the weights: steps of powers of two, float64 sums."""
    import torch

    r = np.random.default_rng(7)
    tokens, top, E, width = 6, 3, 4, 64
    row_of, _ = fast_rows(routing(r, tokens, top, E, "plain"), E)
    y = torch.from_numpy(r.integers(-8, 9, (tokens * top, width)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy((r.integers(1, 9, (tokens, top)) / 8).astype(np.float32)).cuda()
    g = torch.from_numpy(r.integers(-4, 5, (tokens, width)).astype(np.float32)).bfloat16().cuda()
    rows = torch.from_numpy(row_of).cuda()
    gy, gw = torch.zeros_like(y), torch.zeros_like(w)
    L.fp4_moe_combine_backward(g, y, rows, w, gy, gw)

    def value(y, w):
        # (small numbers: the outputs are exact in bf16 where 8 bits hold them, so sums of
        # at most 3 x 8 x 8 eighths are kept below 2^5 with steps of 1/8)
        out = torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda")
        L.fp4_moe_combine(y, rows, w, out)
        return float((out.double() * g.double()).sum()), out

    # by y: one element at a time moves its own output by w
    for row, col in ((0, 0), (5, 17), (tokens * top - 1, width - 1)):
        at = np.argwhere(row_of == row)[0]
        for base in (0.0,):
            lo, hi = torch.zeros_like(y), torch.zeros_like(y)
            lo[row, col], hi[row, col] = base - 1, base + 1
            diff = (value(hi, w)[0] - value(lo, w)[0]) / 2
            assert diff == float(gy[row, col].double()) == float(w[at[0], at[1]] * g[at[0], col].float())
    # by a weight: the others zero, so that outputs are w y with 8 bits at most
    for t, j in ((0, 0), (3, 2), (5, 1)):
        hi, lo = torch.zeros_like(w), torch.zeros_like(w)
        hi[t, j], lo[t, j] = 1.0, -1.0
        assert (value(y, hi)[0] - value(y, lo)[0]) / 2 == float(gw[t, j])


def test_dispatch_gradient_is_combine_without_weights(L):
    import torch

    r = np.random.default_rng(8)
    tokens, top, E, width = 40, 4, 9, 256
    ids = torch.from_numpy(routing(r, tokens, top, E, "padded")).cuda()
    x = torch.zeros(tokens, width, dtype=torch.bfloat16, device="cuda")
    to = torch.zeros(tokens * top, width, dtype=torch.bfloat16, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows = torch.empty_like(ids)
    L.fp4_moe_dispatch(x, ids, E, to, off, rows)
    g = torch.from_numpy(r.integers(-8, 9, (tokens * top, width)).astype(np.float32)).bfloat16().cuda()
    got = torch.empty_like(x)
    L.fp4_moe_combine(g, rows, None, got)
    want = torch.zeros(tokens, width, dtype=torch.float64)
    rc = rows.cpu()
    for j in range(top):
        live = rc[:, j] >= 0
        want[live] += g.cpu().double()[rc[live, j].long()]
    assert torch.equal(got.cpu().double(), want)


def test_layer(L):
    """Dispatch, the grouped FP4 layer on the rows that have an expert, combine: each
    token gets the weighted sum of its experts' layers, as the rows give them."""
    import torch

    r = np.random.default_rng(9)
    tokens, top, E, width, N = 50, 3, 6, 256, 128
    ids = torch.from_numpy(routing(r, tokens, top, E, "padded")).cuda()
    x = torch.from_numpy(r.standard_normal((tokens, width)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy(r.integers(0, 256, (E, N, width // 2)).astype(np.uint8)).cuda()
    sw = torch.full((E, L.fp4_sf_bytes(N, width)), 122, dtype=torch.uint8, device="cuda")
    p = torch.from_numpy(r.random((tokens, top)).astype(np.float32)).cuda()
    rows_max = tokens * top
    to = torch.zeros(rows_max, width, dtype=torch.bfloat16, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows = torch.empty_like(ids)
    y = torch.full((rows_max, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.empty(tokens, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(L.load().fp4_linear_grouped_workspace_size(rows_max, E, width), dtype=torch.uint8, device="cuda")

    def layer():
        L.fp4_moe_dispatch(x, ids, E, to, off, rows)
        L.fp4_linear_grouped(to, off, E, rows_max, w, sw, None, y, N, width, ws)
        L.fp4_moe_combine(y, rows, p, out)

    layer()
    # every row by itself through the dense layer of its expert
    want = torch.zeros(tokens, N, dtype=torch.float64)
    size = torch.zeros(tokens, N, dtype=torch.float64)
    ws1 = torch.zeros(L.fp4_linear_workspace_size(tokens, N, width), dtype=torch.uint8, device="cuda")
    for e in range(E):
        one = torch.empty(tokens, N, dtype=torch.bfloat16, device="cuda")
        L.fp4_linear(x, w[e], sw[e], None, one, tokens, N, width, ws1)
        for j in range(top):
            live = (ids[:, j] == e).cpu()
            part = p.cpu()[live, j].double()[:, None] * one.cpu().double()[live]
            want[live] += part
            size[live] += part.abs()
    # (the dense layer's own sums and rounding may differ in the last place of bf16)
    assert ((out.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -7 + top * 2.0 ** -23) * size).all()
    eager = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


def test_single_token_layer(L):
    """The experts' products of one token, added up: combine with rows in place."""
    import torch

    r = np.random.default_rng(10)
    E, top, width, N = 8, 4, 256, 64
    ids = torch.from_numpy(r.permutation(E)[:top].astype(np.int32)[None]).cuda()
    x = torch.from_numpy(r.standard_normal((1, width)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy(r.integers(0, 256, (E, N, width // 2)).astype(np.uint8)).cuda()
    sw = torch.full((E, L.fp4_sf_bytes(N, width)), 122, dtype=torch.uint8, device="cuda")
    p = torch.from_numpy(r.random((1, top)).astype(np.float32)).cuda()
    y = torch.empty(top, N, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    L.fp4_gemv_mxfp4_experts(x, ids, E, top, top, w, sw, None, y, N, width)
    L.fp4_moe_combine(y, None, p, out)
    ref = (p.cpu().double()[0][:, None] * y.cpu().double()).sum(0)
    size = (p.cpu().double()[0][:, None] * y.cpu().double().abs()).sum(0)
    assert ((out[0].cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + top * 2.0 ** -23 * size).all()
    for j in range(top):
        e = int(ids[0, j])
        one = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
        L.fp4_gemv_mxfp4(x, w[e], sw[e], None, one, 1, N, width)
        assert ((one[0].double() - y[j].double()).abs() <= 2.0 ** -7 * y[j].double().abs() + 2.0 ** -14).all()
