"""Attention of drafted tokens over the MX-quantized cache against the softmax
formula in 64 bits, on the cache's exact values.

Bounds.  A score is a float32 sum of D exact products, at most one ulp each on
magnitudes up to A = scale sum |q k|, and a few roundings of the scaled score:
e = (D + 8) 2^-23 A.  A probability is then off by 2 e + 2^-20 (exponentials,
sums) and, for the second product, by its bf16 rounding 2^-8; the output has
its own bf16 rounding:
  |out - ref| <= 1.01 * 2^-8 |ref| + (2^-8 + 2 e + 2^-19) sum p |v| + T 2^-61
  |lse - ref| <= e + 2^-19 + 2^-22 |ref|
The absolute term: the sums are kept times 2^-64, where float32 ends at 2^-126,
so each of the T terms may lose 2^-62 (twice that with the probability's own)."""
import math

import numpy as np
import pytest

import _layer_ref as R
from _util import bf16_bits_host, bf16_bits_to_f64, dev, host, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


class Problem:
    """Sequences of (context, drafted) lengths over a randomly paged cache."""

    def __init__(self, lens, heads, group, dim, page, fmt, tree=True, seed=0, pages_extra=2, scale_range=(118, 122)):
        import torch

        r = self.r = np.random.default_rng(seed)
        self.lens, self.heads, self.group, self.dim, self.page, self.fmt = lens, heads, group, dim, page, fmt
        per = [-(-(c + n) // page) for c, n in lens]
        pages = sum(per) + pages_extra
        order = r.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(per) + 1), 2 ** 30, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        width = dim if fmt == R.MXFP8 else dim // 2
        self.arrays = []
        lo, hi = scale_range if fmt == R.MXFP8 else (scale_range[0] + 6, scale_range[1] + 6)
        for _ in range(2):
            c = r.integers(0, 256, (pages, heads, page, width)).astype(np.uint8)
            if fmt == R.MXFP8:
                c[(c & 127) == 127] = 0x70
            self.arrays += [c, r.integers(lo, hi, (pages, heads, page, dim // 32)).astype(np.uint8)]
        self.total = sum(n for _, n in lens)
        q = torch.from_numpy(r.standard_normal((self.total, heads * group, dim)).astype(np.float32)).bfloat16()
        self.q = q
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
        self.max_draft = max(n for _, n in lens)
        self.words = -(-self.max_draft // 32)
        self.sees = []
        for c, n in lens:
            s = np.zeros((n, n), bool)
            for j in range(n):
                if tree:
                    if j:
                        s[j] = s[r.integers(0, j)]
                    s[j, j] = True
                else:
                    s[j, :j + 1] = True
            self.sees.append(s)
        self.tree = tree
        self.scale = dim ** -0.5

    def mask_bits(self):
        m = np.zeros((self.total, self.words), np.uint32)
        for b, s in enumerate(self.sees):
            for i in range(len(s)):
                for j in np.flatnonzero(s[i]):
                    m[self.cu[b] + i, j // 32] |= np.uint32(1 << (j % 32))
        return m

    def run(self, L, max_seq=None, stream=None, out=None):
        import torch

        self.dev = [dev(a) for a in self.arrays]
        cache = L.kv_cache(*self.dev, self.page, self.fmt)
        q = self.q.cuda()
        out = torch.full_like(q, float("nan")) if out is None else out
        lse = torch.full((self.total, self.heads * self.group), float("nan"), device="cuda")
        max_seq = max_seq or max(c + n for c, n in self.lens)
        need = L.fp4_kv_attention_workspace_size(len(self.lens), self.total, self.heads * self.group, self.heads, self.dim,
                                                 max_seq, self.max_draft)
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        mask = dev(self.mask_bits().view(np.int32)) if self.tree else None
        ctx = dev(np.array([c for c, _ in self.lens], np.int32))
        L.fp4_kv_attention(cache, q, out, dev(self.table), ctx, dev(self.cu), max_seq, self.max_draft, ws, tree_mask=mask,
                           lse=lse, softmax_scale=self.scale)
        return bf16_bits_to_f64(bf16_bits_host(out)), host(lse).astype(np.float64)

    def check(self, out, lse):
        q = self.q.double().numpy()
        for b, (ctx, n) in enumerate(self.lens):
            if n == 0:
                continue
            t = np.arange(ctx + n)
            pg, sl = self.table[b, t // self.page], t % self.page
            k, v = (R.mx_values(R.unpack(self.arrays[2 * i][pg, :, sl], self.fmt), self.arrays[2 * i + 1][pg, :, sl], self.fmt)
                    for i in range(2))
            sees = np.concatenate((np.ones((n, ctx), bool), self.sees[b]), 1)
            rows = np.s_[self.cu[b]:self.cu[b] + n]
            for h in range(self.heads * self.group):
                ref, rl, absv, mag = R.attend(q[rows, h], k[:, h // self.group], v[:, h // self.group], sees, self.scale)
                e = (self.dim + 8) * 2.0 ** -23 * mag
                got, gl = out[rows, h], lse[rows, h]
                bound = 1.01 * 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -19) * absv + (ctx + n) * 2.0 ** -61
                nan = np.isnan(ref)
                assert np.array_equal(np.isnan(got), nan)
                assert np.all((np.abs(got - ref) <= bound)[~nan]), (b, h, np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-30)))
                none = ~sees.any(1)
                assert np.all(np.isneginf(gl[none])) and not got[none].any()
                fine = ~none & ~np.isnan(rl)
                assert np.all(np.abs(gl[fine] - rl[fine]) <= e[fine] + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl[fine]))


LENS = [[(0, 1)], [(1, 1)], [(15, 1), (16, 1), (17, 1)], [(503, 1)], [(40, 5), (0, 3), (131, 1), (64, 0), (7, 6)],
        [(300, 17), (0, 33)], [(1100, 64)], [(2500, 2), (30, 1)]]


@pytest.mark.parametrize("lens", LENS, ids=lambda l: "-".join("%d+%d" % x for x in l))
@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("heads,group,dim,page", [(2, 4, 128, 16), (1, 1, 64, 48), (3, 7, 128, 64), (2, 8, 64, 32)])
@pytest.mark.parametrize("tree", [False, True])
def test_matches_the_formula(L, lens, fmt, heads, group, dim, page, tree):
    p = Problem(lens, heads, group, dim, page, fmt, tree, seed=len(lens) + dim)
    p.check(*p.run(L))
    assert L.fp4_get_device_status() == 0


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_split_contexts_give_the_same(L, fmt):
    """A long sequence split over many CTAs, with ragged others; a looser bound of
    the lengths changes the cut but not the result's error."""
    p = Problem([(9001, 3), (17, 2), (4000, 3)], 2, 4, 128, 64, fmt, seed=5)
    a = p.run(L)
    p.check(*a)
    b = p.run(L, max_seq=100000)
    p.check(*b)
    again = p.run(L)
    assert np.array_equal(a[0], again[0]) and np.array_equal(a[1], again[1])


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("group", [2, 16])
def test_rows_without_a_visible_token(L, fmt, group):
    p = Problem([(0, 4), (70, 4)], 2, group, 64, 16, fmt, seed=6)
    p.sees[0][2] = False
    p.sees[1][3] = False          # still sees its context
    p.sees[0][0] = False
    p.check(*p.run(L))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
@pytest.mark.parametrize("group,draft", [(2, 5), (8, 9)])
def test_nan_reaches_only_the_rows_that_see_it(L, fmt, group, draft):
    p = Problem([(50, draft), (20, 3)], 2, group, 128, 16, fmt, seed=7)
    pos = 50 + 2                                            # a drafted token that siblings do not see
    for a in (1, 3):
        p.arrays[a][p.table[0, pos // 16], 1, pos % 16, a - 1] = 255
    p.arrays[3][p.table[0, (50 + 4) // 16], 0, (50 + 4) % 16, 1] = 255
    tail = 50 + draft                                       # past the end, in the last page
    if tail % 16:
        p.arrays[1][p.table[0, tail // 16], :, tail % 16] = 255
        p.arrays[3][p.table[0, tail // 16], :, tail % 16] = 255
    out, lse = p.run(L)
    p.check(out, lse)
    assert np.isnan(out).any() and not np.isnan(out).all()


def test_nan_in_the_context_reaches_every_row(L):
    p = Problem([(200, 3)], 1, 4, 64, 16, R.MXFP8, seed=8)
    p.arrays[3][p.table[0, 100 // 16], 0, 100 % 16, 1] = 255
    out, _ = p.run(L)
    assert np.isnan(out[:, :, 32:]).all() and not np.isnan(out[:, :, :32]).any()


@pytest.mark.parametrize("fmt,scales", [(R.MXFP8, (60, 66)), (R.MXFP8, (176, 180)), (R.MXFP4, (60, 66)), (R.MXFP4, (176, 180))])
def test_small_and_large_magnitudes(L, fmt, scales):
    """Values around 2^-60 and 2^55: softmax is flat or one-hot, the output keeps the scale."""
    p = Problem([(150, 2)], 1, 4, 64, 16, fmt, seed=9, scale_range=scales)
    if scales[0] > 100:
        p.arrays[1][:] = 120                                # ordinary keys, large values
    p.check(*p.run(L))


def test_large_scores_stay_finite(L):
    p = Problem([(700, 2)], 1, 4, 128, 16, R.MXFP8, seed=10, scale_range=(126, 130))
    out, lse = p.run(L)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    p.check(out, lse)


def test_strided_queries_and_another_stream(L):
    import torch

    p = Problem([(90, 3), (10, 2)], 2, 4, 64, 16, R.MXFP8, seed=11)
    want = p.run(L)
    wide = torch.randn(p.total, 3 * 8 * 64 + 8, device="cuda").bfloat16()
    wide[:, :8 * 64] = p.q.cuda().flatten(1)
    q = wide[:, :8 * 64].unflatten(1, (8, 64))
    back = torch.zeros(8, p.total, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    cache = L.kv_cache(*p.dev, p.page, p.fmt)
    ctx, mask = dev(np.array([90, 10], np.int32)), dev(p.mask_bits().view(np.int32))
    table, cu = dev(p.table), dev(p.cu)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.fp4_kv_attention(cache, q, back.transpose(0, 1), table, ctx, cu, 93, 3, None, tree_mask=mask,
                           softmax_scale=p.scale)
    torch.cuda.current_stream().wait_stream(side)
    assert np.array_equal(bf16_bits_to_f64(bf16_bits_host(back.transpose(0, 1).contiguous())), want[0])


def test_offsets_past_32_bits(L):
    """Pages at the end of a cache whose arrays pass 4 GB."""
    import torch

    p = Problem([(200, 2)], 8, 2, 128, 64, R.MXFP8, seed=12, pages_extra=0)
    pages = (1 << 32) // (8 * 64 * 128) + 8
    small = p.arrays
    big = [torch.empty((pages, *a.shape[1:]), dtype=torch.uint8, device="cuda") for a in small]
    for t, a in zip(big, small):
        t[-len(a):] = dev(a)
    cache = L.kv_cache(*big, 64, R.MXFP8)
    table = p.table.copy()
    table[table < 2 ** 30] += pages - len(small[0])
    q = p.q.cuda()
    out = torch.empty_like(q)
    lse = torch.empty(p.total, 16, device="cuda")
    L.fp4_kv_attention(cache, q, out, dev(table), dev(np.array([200], np.int32)), dev(p.cu), 202, 2, None,
                       tree_mask=dev(p.mask_bits().view(np.int32)), lse=lse)
    p.check(bf16_bits_to_f64(bf16_bits_host(out)), host(lse).astype(np.float64))


def test_appended_tokens_are_attended(L):
    """Append with rotation, then attention over what was appended: one decode step."""
    import torch

    r = np.random.default_rng(13)
    heads, group, dim, page, T = 2, 4, 128, 16, 37
    kv = torch.from_numpy(r.standard_normal((2, T, heads, dim)).astype(np.float32)).bfloat16().cuda()
    p = Problem([(T - 1, 1)], heads, group, dim, page, R.MXFP4, tree=False, seed=14)
    p.dev = [dev(a) for a in p.arrays]
    cache = L.kv_cache(*p.dev, page, R.MXFP4)
    t = np.arange(T)
    slots = p.table[0, t // page].astype(np.int64) * page + t % page
    table = torch.empty(64, dim, device="cuda")
    L.fp4_rope_table(table, 64, dim, 10000.0)
    L.fp4_kv_append(cache, kv[0], kv[1], dev(slots), rope=L.rope_params(table, dim), positions=dev(t.astype(np.int32)))
    q = p.q.cuda()
    out, lse = torch.empty_like(q), torch.empty(1, heads * group, device="cuda")
    L.fp4_kv_attention(cache, q, out, dev(p.table), dev(np.array([T - 1], np.int32)), dev(p.cu), T, 1, None, lse=lse)
    p.arrays = [host(a) for a in p.dev]
    p.check(bf16_bits_to_f64(bf16_bits_host(out)), host(lse).astype(np.float64))
