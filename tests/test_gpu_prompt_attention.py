"""Attention over whole prompts against the softmax formula in 64 bits.

Bounds.  A score is a float32 sum of D exact products, at most one ulp each on
magnitudes up to A = scale sum |q k|, and a few roundings of the scaled score:
e = (D + 8) 2^-23 A.  A weight is then off by 2 e + 2^-20 (exponentials, sums) and,
for the product with v, by its bf16 rounding 2^-8; the output has its own:
  |out - ref| <= 1.01 * 2^-8 |ref| + (2^-8 + 2 e + 2^-19) sum p |v| + 2^-133
  |lse - ref| <= e + 2^-19 + 2^-22 |ref|"""
import numpy as np
import pytest

from _util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def normal(r, *shape):
    import torch

    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).bfloat16()


def offsets(lens):
    import torch

    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def reference(q, k, v, lens, causal, scale):
    """out, lse, sum p |v|, bound of the score magnitudes, by sequence and head."""
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    heads, group = k.shape[1], q.shape[1] // k.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    lse, mag = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    row = at = 0
    for n, m in lens:
        seen = np.ones((n, m), bool)
        if causal:
            seen = np.arange(m)[None] <= np.arange(n)[:, None] + (m - n)
        for h in range(heads * group if n and m else 0):
            qq, kk, vv = q[row:row + n, h], k[at:at + m, h // group], v[at:at + m, h // group]
            with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
                x = np.where(seen, qq @ kk.T * scale, -np.inf)
                mx = x.max(-1)
                mx = np.where(np.isneginf(mx), 0.0, mx)
                p = np.where(seen, np.exp(x - mx[:, None]), 0.0)
                total = p.sum(-1)
                w = np.where(total[:, None] == 0, 0.0, p / total[:, None])
                lse[row:row + n, h] = mx + np.log(total)
                if np.isfinite(vv).all():
                    out[row:row + n, h], size[row:row + n, h] = w @ vv, w @ np.abs(vv)
                else:
                    for i in range(n):
                        out[row + i, h] = w[i, seen[i]] @ vv[seen[i]]
                        size[row + i, h] = w[i, seen[i]] @ np.abs(vv[seen[i]])
                mag[row:row + n, h] = np.where(seen, np.abs(qq) @ np.abs(kk).T * scale, 0.0).max(-1)
        row, at = row + n, at + m
    return out, lse, size, mag


def check(out, lse, ref, dim):
    want, want_lse, size, mag = ref
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        e = ((dim + 8) * 2.0 ** -23 * mag)[..., None]
        bound = 1.01 * 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * e + 2.0 ** -19) * size + 2.0 ** -133
        assert np.array_equal(np.isnan(out), np.isnan(want))
        inf = np.isinf(want)
        assert np.array_equal(out[inf], want[inf])
        ok = np.isfinite(want)
        assert (np.abs(out - want)[ok] <= bound[ok]).all(), float((np.abs(out - want)[ok] / bound[ok]).max())
        ok = np.isfinite(want_lse)
        assert np.array_equal(lse[~ok], want_lse[~ok], equal_nan=True)
        assert (np.abs(lse - want_lse)[ok] <= (e[..., 0] + 2.0 ** -19 + 2.0 ** -22 * np.abs(want_lse))[ok]).all()


class Problem:
    def __init__(self, lens, heads, group, dim, seed=0, layout="rows", extra=3):
        import torch

        r = np.random.default_rng(seed)
        self.lens, self.dim = lens, dim
        n, m = sum(a for a, _ in lens), sum(b for _, b in lens)
        self.q = normal(r, n + extra, heads * group, dim).cuda()
        if layout == "rows":     # slices of one projection's rows
            kv = normal(r, m + extra, 2 * heads, dim).cuda()
            self.k, self.v = kv[:, :heads], kv[:, heads:]
            self.out = torch.full_like(self.q, 7.0)
        else:                    # heads outermost, gaps between them
            self.k = normal(r, heads, m + extra + 5, dim).cuda().transpose(0, 1)[5:]
            self.v = normal(r, heads, m + extra, dim + 8).cuda().transpose(0, 1)[..., :dim]
            self.q = self.q.transpose(0, 1).contiguous().transpose(0, 1)
            self.out = torch.full((heads * group, n + extra, dim + 16), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., 8:8 + dim]
        self.lse = torch.full((n + extra, heads * group), 7.0, dtype=torch.float32, device="cuda")
        self.n, self.m = n, m
        self.cu, self.cu_k = offsets([a for a, _ in lens]), offsets([b for _, b in lens])

    def workspace(self, L):
        import torch

        need = L.fp4_prompt_attention_workspace_size(len(self.lens), self.q.shape[0], self.k.shape[0], self.q.shape[1],
                                                     self.k.shape[1], self.dim)
        return torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def run(self, L, causal=True, scale=None, ws=None, **kw):
        L.fp4_prompt_attention(self.q, self.k, self.v, self.out, self.cu, self.cu_k, self.workspace(L) if ws is None else ws,
                               causal=causal, lse=self.lse, softmax_scale=scale, **kw)

    def check(self, causal=True, scale=None):
        # rows behind the last sequence are as they were
        assert (self.out[self.n:] == 7.0).all() and (self.lse[self.n:] == 7.0).all()
        ref = reference(self.q[:self.n], self.k[:self.m], self.v[:self.m], self.lens, causal,
                        float(np.float32(self.dim ** -0.5 if scale is None else scale)))
        check(self.out[:self.n], self.lse[:self.n], ref, self.dim)


LENS = [
    [(1, 1)], [(1, 300)], [(5, 0)], [(128, 128)], [(129, 129)], [(257, 257)], [(100, 357)], [(300, 100)], [(64, 1000)],
    [(0, 0), (3, 3), (0, 7), (129, 129), (1, 1), (2, 1), (40, 513), (0, 0)],
    [(7, 7)] * 40, [(600, 600), (1, 1), (383, 383)], [(1, 5000), (1, 1), (3, 2111)],
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,group,dim,layout", [(1, 1, 64, "rows"), (2, 4, 128, "rows"), (3, 3, 128, "heads"), (2, 8, 64, "heads"),
                                                    (1, 5, 128, "rows")])
@pytest.mark.parametrize("lens", LENS)
def test_formula(L, lens, heads, group, dim, layout, causal):
    p = Problem(lens, heads, group, dim, seed=len(lens) + dim + group, layout=layout)
    p.run(L, causal)
    p.check(causal)


@pytest.mark.parametrize("heads,group,dim", [(2, 130, 64), (1, 256, 128), (1, 100, 64), (2, 17, 128)])
def test_many_heads(L, heads, group, dim):
    """More query heads of a key head than a tile has rows, and groups that leave rows over."""
    for causal in (True, False):
        p = Problem([(3, 3), (1, 140), (9, 4)], heads, group, dim, seed=group)
        p.run(L, causal)
        p.check(causal)


def test_one_key_head_of_many_sequences(L):
    """More sequences than a block has threads, empty ones among them."""
    lens = [((i * 7) % 5, (i * 7) % 5 + (i % 3)) if i % 4 else (0, 2) for i in range(700)]
    p = Problem(lens, 1, 2, 64, seed=11)
    p.run(L)
    p.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_long_prompt(L, dim):
    """A prompt of many tiles; rows spread over it against the formula."""
    import torch

    n, heads, group = 9001, 2, 2
    p = Problem([(n, n)], heads, group, dim, seed=dim)
    p.run(L)
    q, k, v = (x.double() for x in (p.q, p.k, p.v))
    for i in (0, 1, 127, 128, 511, 4095, 4096, 6000, n - 1):
        for h in range(heads * group):
            x = k[:i + 1, h // group] @ q[i, h] * dim ** -0.5
            w = torch.softmax(x, 0)
            ref, size = w @ v[:i + 1, h // group], w @ v[:i + 1, h // group].abs()
            e = (dim + 8) * 2.0 ** -23 * float((k[:i + 1, h // group].abs() @ q[i, h].abs()).max()) * dim ** -0.5
            assert ((p.out[i, h].double() - ref).abs() <= 1.01 * 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e + 2.0 ** -19) * size).all()
            want = float(torch.logsumexp(x, 0))
            assert abs(float(p.lse[i, h]) - want) <= e + 2.0 ** -19 + 2.0 ** -22 * abs(want)
    assert (p.out[n:] == 7.0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [[(200, 200), (70, 300)], [(130, 100)]])
def test_nan_where_it_is_not_seen(L, lens, dim):
    """NaN and Inf in keys and values reach exactly the queries that see them; so do
    those behind the last sequence, which nobody sees."""
    p = Problem(lens, 2, 2, dim, seed=3)
    nan, inf = float("nan"), float("inf")
    p.k[p.m:], p.v[p.m:] = nan, nan
    m0 = lens[0][1]
    p.v[m0 - 1, 0, 3] = nan           # seen by the last query of the first sequence
    p.v[m0 - 40, 1, 5] = inf
    p.v[m0 - 41, 1, 6] = -inf
    p.v[m0 - 20, 1, 6] = inf          # with the one above: NaN
    p.k[m0 - 3, 0, 7] = nan
    p.q[2, 1, 0] = nan
    if len(lens) > 1:
        p.v[m0 + 299, 1] = inf
        p.v[m0 + 250, 0, 9] = nan
    p.run(L)
    p.check()


def test_scores_far_apart(L):
    """Rows whose largest score comes last, far above the others, and scores of
    thousands: the running maximum moves."""
    import torch

    p = Problem([(700, 700)], 1, 2, 64, seed=4)
    p.k *= torch.linspace(0.01, 40.0, p.k.shape[0]).cuda()[:, None, None].to(p.k)
    p.run(L, scale=1.0)
    p.check(scale=1.0)


def test_all_scores_equal(L):
    p = Problem([(300, 300)], 2, 1, 128, seed=5)
    p.q.zero_()
    p.run(L)
    p.check()


def test_without_lse_and_keys(L):
    import torch

    p = Problem([(4, 0), (130, 0)], 2, 2, 64, seed=6, extra=0)
    assert p.k.shape[0] == 0
    L.fp4_prompt_attention(p.q, p.k, p.v, p.out, p.cu, p.cu_k, p.workspace(L))
    assert (p.out == 0).all()
    p = Problem([(150, 150)], 2, 2, 64, seed=6)
    p.run(L)
    out = p.out.clone()
    p.out.fill_(7.0)
    L.fp4_prompt_attention(p.q, p.k, p.v, p.out, p.cu, None, p.workspace(L))
    assert torch.equal(p.out, out)


def test_offsets_out_of_order(L):
    """Wrong offsets are clamped: the call ends and writes nothing outside."""
    import torch

    p = Problem([(100, 100)], 1, 2, 64, seed=7)
    p.cu = torch.tensor([0, 200, -5, 60, 2 ** 30], dtype=torch.int32, device="cuda")
    p.cu_k = torch.tensor([0, 2 ** 31 - 1, 50, -7, 90], dtype=torch.int32, device="cuda")
    p.lens = [(1, 1)] * 4
    p.run(L)
    torch.cuda.synchronize()
    assert L.fp4_get_device_status() == 0


def test_repeats_streams_and_graphs(L):
    """The same bits again, on another stream, and from two graphs that share a workspace."""
    import torch

    p = Problem([(400, 400), (33, 700), (1, 1)], 2, 4, 128, seed=8)
    ws = p.workspace(L)
    p.run(L, ws=ws)
    first = p.out.clone(), p.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.out.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.run(L, ws=ws)
    side.synchronize()
    assert torch.equal(p.out, first[0]) and torch.equal(p.lse, first[1])
    o = Problem([(90, 90)], 1, 1, 64, seed=9)
    graphs = []
    for x in (p, o):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(L, ws=ws if x is p else ws[: max(o.workspace(L).numel(), 1)])
        graphs.append(g)
    for _ in range(3):
        p.out.fill_(7.0)
        o.out.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first[0]) and torch.equal(p.lse, first[1])
        o.check()
