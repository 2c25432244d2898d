"""The decoder layer's operators as a program calls them: two calls at once on two
streams, calls of several launches in graphs, inputs that are broadcast, many narrow
pairs.  Every call gives the bits that it gives alone."""
import numpy as np
import pytest

from _util import dev, lib
from test_gpu_gemv import acts, check, swizzle, weight
from test_gpu_moe import fast_rows, routing
from test_gpu_prompt_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def test_prompts_on_two_streams(L):
    """Calls with workspaces of their own, cut units and whole ones, at the same time."""
    import torch

    sides = []
    for lens, heads, group, dim in (([(2500, 2500)], 2, 4, 128), ([(90, 1400)] * 9, 2, 2, 64)):
        p = Problem(lens, heads, group, dim, seed=dim)
        ws = p.workspace(L)
        p.run(L, ws=ws)
        p.check()
        sides.append((p, ws, p.out.clone(), p.lse.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for p, *_ in sides:
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for p, ws, _, _, stream in sides:
            with torch.cuda.stream(stream):
                p.run(L, ws=ws)
    torch.cuda.synchronize()
    assert L.fp4_get_device_status() == 0
    for p, _, out, lse, _ in sides:
        assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


def experts_layer(L, seed, tokens, top, E, n, k):
    """A call of a MoE layer's products and sums without sorting, and its output."""
    import torch

    r = np.random.default_rng(seed)
    parts = [weight(r, n, k, False) for _ in range(E)]
    w = torch.stack([dev(c) for c, _, _ in parts])
    sw = torch.stack([dev(swizzle(s)) for _, s, _ in parts])
    ids, x = dev(routing(r, tokens, top, E, "plain")), acts(r, tokens, k).cuda()
    p = dev(r.random((tokens, top)).astype(np.float32))
    y = torch.empty(tokens * top, n, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")

    def call():
        L.fp4_gemv_mxfp4_experts(x, ids, E, tokens * top, top, w, sw, None, y, n, k)
        L.fp4_moe_combine(y, None, p, out)

    return call, out


def test_products_on_two_streams(L):
    import torch

    r = np.random.default_rng(3)
    m, n, k = 5, 3000, 2080
    codes, s, w = weight(r, n, k, True)
    x, dense = acts(r, m, k), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    args = (x.cuda(), dev(codes), dev(swizzle(s)), 1.0, None, dense, m, n, k)
    moe, out = experts_layer(L, 4, 3, 4, 8, 520, 1024)
    calls = (lambda: L.fp4_gemv_nvfp4(*args), moe)
    for c in calls:
        c()
    check(dense, x, w, None)
    alone = dense.clone(), out.clone()
    torch.cuda.synchronize()
    dense.zero_()
    out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(300):
        for c, stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                c()
    torch.cuda.synchronize()
    assert L.fp4_get_device_status() == 0
    assert torch.equal(dense, alone[0]) and torch.equal(out, alone[1])


# (activations of K elements that leave room for a few tokens of a launch)
@pytest.mark.parametrize("m,n,k", [(8, 300, 65536), (7, 1000, 20000), (8, 130, 16416)])
@pytest.mark.parametrize("nv", [False, True])
def test_products_of_several_launches_again_and_in_a_graph(L, m, n, k, nv):
    import torch

    r = np.random.default_rng(n)
    codes, s, w = weight(r, n, k, nv)
    x, out = acts(r, m, k), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    args = (x.cuda(), dev(codes), dev(swizzle(s))) + ((1.0,) if nv else ()) + (None, out, m, n, k)
    call = L.fp4_gemv_nvfp4 if nv else L.fp4_gemv_mxfp4
    call(*args)
    check(out, x, w, None)
    first = out.clone()
    for _ in range(200):
        call(*args)
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*args)
        call(*args)
    for _ in range(20):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    assert L.fp4_get_device_status() == 0


def test_broadcast_inputs(L):
    """One token's vector, or one gradient, for all tokens (a row stride of zero)."""
    import torch

    r = np.random.default_rng(5)
    tokens, top, E, width = 400, 3, 11, 72
    ids = routing(r, tokens, top, E, "padded")
    row_of, offsets = fast_rows(ids, E)
    v = torch.from_numpy(r.standard_normal((1, width)).astype(np.float32)).bfloat16().cuda()
    to = torch.full((tokens * top, width), 7.0, dtype=torch.bfloat16, device="cuda")
    off, rows = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(tokens, top, dtype=torch.int32, device="cuda")
    L.fp4_moe_dispatch(v.expand(tokens, width), dev(ids), E, to, off, rows)
    assert np.array_equal(rows.cpu().numpy(), row_of) and np.array_equal(off.cpu().numpy(), offsets)
    assert (to[:offsets[-1]] == v).all() and (to[offsets[-1]:] == 7.0).all()
    w = dev(r.random((tokens, top)).astype(np.float32))
    got, want = (torch.full((tokens * top, width), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gw, ww = torch.empty_like(w), torch.empty_like(w)
    L.fp4_moe_combine_backward(v.expand(tokens, width), to, rows, w, got, gw)
    L.fp4_moe_combine_backward(v.expand(tokens, width).contiguous(), to, rows, w, want, ww)
    assert torch.equal(got, want) and torch.equal(gw, ww)


def test_a_million_narrow_pairs(L):
    import torch

    r = np.random.default_rng(6)
    tokens, top, E, width = 131075, 8, 1024, 8
    ids = routing(r, tokens, top, E, "padded")
    x = torch.from_numpy(r.standard_normal((tokens, width)).astype(np.float32)).bfloat16().cuda()
    to = torch.full((tokens * top, width), 7.0, dtype=torch.bfloat16, device="cuda")
    off, rows = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(tokens, top, dtype=torch.int32, device="cuda")
    L.fp4_moe_dispatch(x, dev(ids), E, to, off, rows)
    row_of, offsets = fast_rows(ids, E)
    assert np.array_equal(rows.cpu().numpy(), row_of) and np.array_equal(off.cpu().numpy(), offsets)
    t, j = np.nonzero(row_of >= 0)
    assert torch.equal(to[torch.from_numpy(row_of[t, j]).long().cuda()], x[torch.from_numpy(t).cuda()])


def test_dispatch_in_a_graph_and_on_two_streams(L):
    """The sort over a cluster with the copies behind it, where the call before them in
    the graph has only just written the vectors."""
    import torch

    r = np.random.default_rng(7)
    tokens, top, E, width = 3001, 4, 1024, 264
    sources = [torch.from_numpy(r.standard_normal((tokens, width)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    routes = [dev(routing(r, tokens, top, E, "padded")) for _ in range(2)]

    def buffers():
        return (torch.empty(tokens * top, width, dtype=torch.bfloat16, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                torch.empty(tokens, top, dtype=torch.int32, device="cuda"))

    def right(x, ids, to, off, rows):
        row_of, offsets = fast_rows(ids.cpu().numpy(), E)
        assert np.array_equal(rows.cpu().numpy(), row_of) and np.array_equal(off.cpu().numpy(), offsets)
        t, j = np.nonzero(row_of >= 0)
        assert torch.equal(to[torch.from_numpy(row_of[t, j]).long().cuda()], x[torch.from_numpy(t).cuda()])

    x, ids, src, src_ids = torch.empty_like(sources[0]), torch.empty_like(routes[0]), torch.empty_like(sources[0]), torch.empty_like(routes[0])
    got = buffers()
    src.copy_(sources[0])
    src_ids.copy_(routes[0])
    L.fp4_moe_dispatch(sources[0], routes[0], E, *got)
    right(sources[0], routes[0], *got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(src)
        ids.copy_(src_ids)
        L.fp4_moe_dispatch(x, ids, E, *got)
    for i in range(30):
        src.copy_(sources[i % 2])
        src_ids.copy_(routes[i % 2])
        graph.replay()
        if i % 2 or i == 0:
            right(sources[i % 2], routes[i % 2], *got)
    both = [buffers() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(100):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                L.fp4_moe_dispatch(sources[i], routes[i], E, *both[i])
    torch.cuda.synchronize()
    for i in range(2):
        right(sources[i], routes[i], *both[i])


def test_most_sequences(L):
    """65535 sequences, nearly all of them empty or of a token or two."""
    n = np.zeros(65535, np.int64)
    n[::9], n[4::31], n[65534], n[30000] = 1, 2, 300, 700
    m = n + (np.arange(65535) % 3) * (n > 0)
    p = Problem(list(zip(n.tolist(), m.tolist())), 1, 2, 64, seed=8)
    p.run(L)
    p.check()
    assert L.fp4_get_device_status() == 0


def test_offsets_past_32_bits(L):
    """Token strides that bring the last rows more than 2^31 elements in, for every operator
    that takes strides."""
    import torch

    r = np.random.default_rng(9)
    T, wide, heads, dim = 2200, 1 << 20, 2, 64
    base = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    assert (T - 1) * wide > 2 ** 31

    def place(k, n):
        return base[:, 4096 * k:4096 * k + n]

    p = Problem([(T, T)], heads, 2, dim, seed=9, extra=0)
    p.run(L)
    p.check()
    out, lse = p.out.clone(), p.lse.clone()
    for i, name in enumerate(("q", "k", "v", "out")):
        t = getattr(p, name)
        far = place(i, t.shape[1] * dim).unflatten(1, (t.shape[1], dim))
        far.copy_(t)
        setattr(p, name, far)
    p.out.fill_(7.0)
    p.run(L)
    assert torch.equal(p.out, out) and torch.equal(p.lse, lse)
    # norms of heads
    w = torch.from_numpy(r.standard_normal(dim).astype(np.float32)).bfloat16().cuda()
    near = [torch.empty(T, h, dim, dtype=torch.bfloat16, device="cuda") for h in (4, 2)]
    L.fp4_qk_norm_rope(p.q.contiguous(), p.k.contiguous(), *near, w, w)
    far = [place(4, 4 * dim).unflatten(1, (4, dim)), place(5, 2 * dim).unflatten(1, (2, dim))]
    L.fp4_qk_norm_rope(p.q, p.k, *far, w, w)
    assert all(torch.equal(a, b) for a, b in zip(near, far))
    # experts' rows and back
    x, top, E = place(0, 256), 2, 7
    ids = dev(routing(r, T, top, E, "plain"))
    to, want = (torch.empty(T * top, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off, rows = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T, top, dtype=torch.int32, device="cuda")
    L.fp4_moe_dispatch(x.contiguous(), ids, E, want, off, rows)
    L.fp4_moe_dispatch(x, ids, E, to, off, rows)
    assert torch.equal(to, want)
    p2 = dev(r.random((T, top)).astype(np.float32))
    near = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
    L.fp4_moe_combine(to, rows, p2, near)
    L.fp4_moe_combine(to, rows, p2, place(6, 256))
    assert torch.equal(near, place(6, 256))
    a, b = torch.empty_like(to), torch.empty_like(to)
    ga, gb = torch.empty_like(p2), torch.empty_like(p2)
    L.fp4_moe_combine_backward(near, to, rows, p2, a, ga)
    L.fp4_moe_combine_backward(place(6, 256), to, rows, p2, b, gb)
    assert torch.equal(a, b) and torch.equal(ga, gb)


def test_experts_past_32_bits(L):
    """Weights of more than 2^32 bytes: the last experts' rows against their own products."""
    import torch

    E, n, k = 300, 8200, 4096
    g = torch.Generator(device="cuda").manual_seed(10)
    w = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    sw = torch.randint(118, 124, (E, L.fp4_sf_bytes(n, k)), dtype=torch.uint8, device="cuda", generator=g)
    assert w.numel() > 2 ** 32
    r = np.random.default_rng(10)
    ids = np.array([E - 1, 0, E - 2, 255], np.int32)
    x = acts(r, 1, k).cuda()
    out = torch.empty(4, n, dtype=torch.bfloat16, device="cuda")
    L.fp4_gemv_mxfp4_experts(x, dev(ids), E, 4, 4, w, sw, None, out, n, k)
    one, size = torch.empty(1, n, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    for i, e in enumerate(ids):
        L.fp4_gemv_mxfp4(x, w[e], sw[e], None, one, 1, n, k)
        L.fp4_gemv_mxfp4(x.abs(), w[e] & 0x77, sw[e], None, size, 1, n, k)    # sums of magnitudes
        # (the same products summed in another order, and two roundings)
        assert ((out[i].double() - one[0].double()).abs() <= 2.0 ** -7 * one[0].double().abs()
                + 1.01 * 2 * (k / 16 + 40) * 2.0 ** -23 * size[0].double()).all()
