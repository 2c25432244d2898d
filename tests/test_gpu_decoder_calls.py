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
