"""The FP8 linear layer with a scale per block of 128 on the GPU against its
formula in 64 bits.

Quantizers: every code and scale bit-exact (one IEEE float32 operation at a
time).  GEMM, with the kernel's own operands decoded exactly: one bf16
rounding (2^-8 relative), and at most one float32 ulp per addition of the 128
products of a block and of the block sums, on magnitudes up to sum |a b|:
|out - ref| <= 1.01 * 2^-8 |ref| + (128 + blocks + 8) 2^-23 sum |a b|."""
import numpy as np
import pytest

import _layer_ref as R
from _util import bf16_bits_host, bf16_bits_to_f64, dev, dev_bf16, host, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def _bf16(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def _quant_act(L, bits):
    import torch

    M, K = bits.shape
    codes = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    kb, mp = -(-K // 128), -(-M // 4) * 4
    assert L.fp4_fp8_act_scale_bytes(M, K) == kb * mp * 4
    scales = torch.full((kb, mp), -1.0, dtype=torch.float32, device="cuda")
    L.fp4_quant_act_fp8_b128(dev_bf16(bits), codes, scales, M, K)
    return codes, scales


def _check(out_bits, xv, wv, bias, kb):
    ref = xv @ wv.T
    mag = np.abs(xv) @ np.abs(wv).T
    if bias is not None:
        b = bf16_bits_to_f64(bias)
        ref, mag = ref + b, mag + np.abs(b)
    err = np.abs(bf16_bits_to_f64(out_bits) - ref)
    bound = 1.01 * 2.0 ** -8 * np.abs(ref) + (128 + kb + 8) * 2.0 ** -23 * mag
    assert np.all(err <= bound), f"max err/bound = {np.max(err / np.maximum(bound, 1e-300))}"


@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 272), (130, 400), (33, 1024)])
def test_activation_quantizer_is_exact(L, M, K):
    r = np.random.default_rng(M * K)
    x = r.standard_normal((M, K)) * np.exp(r.uniform(-8, 8, (M, 1)))
    x[0, :128] = 0
    if M > 2:
        x[1, 5], x[2, 7] = np.inf, np.nan
    bits = _bf16(x)
    if M > 4:
        bits[4, :128] = 3                   # subnormals only
    codes, scales = _quant_act(L, bits)
    xv = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    want, ws = R.fp8_quantize(xv, 1)
    assert np.array_equal(host(codes), want)
    assert np.array_equal(host(scales)[:, :M].T, ws, equal_nan=True)


@pytest.mark.parametrize("N,K", [(8, 16), (136, 272), (256, 384), (1000, 144)])
def test_weight_quantizer_is_exact(L, N, K):
    import torch

    r = np.random.default_rng(N + K)
    w = r.standard_normal((N, K)) * 0.02
    if N > 128:
        w[130, 3] = np.nan
    bits = _bf16(w)
    codes = torch.full((N, K), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-N // 128), -(-K // 128)), -1.0, dtype=torch.float32, device="cuda")
    L.fp4_quant_weight_fp8_b128(dev_bf16(bits), codes, scales, N, K)
    want, ws = R.fp8_quantize((bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64), 128)
    assert np.array_equal(host(codes), want)
    assert np.array_equal(host(scales), ws, equal_nan=True)


SHAPES = [(1, 8, 16), (1, 4096, 4096), (7, 136, 272), (16, 128, 128), (17, 264, 1040), (33, 1000, 400), (64, 2048, 1024),
          (65, 520, 640), (128, 384, 2048), (129, 256, 528), (300, 1032, 784), (515, 1288, 1296), (1024, 2048, 256),
          (2041, 1032, 400)]
# problems with many 256 x 256 tiles (CTA pairs): odd rows, short last blocks, N ends inside a tile
SHAPES += [(300, 5128, 1040), (1500, 2056, 272), (129, 9736, 144), (2048, 2048, 384)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_linear_matches_the_formula(L, M, N, K, with_bias):
    import torch

    r = np.random.default_rng(M + N + K)
    x = r.standard_normal((M, K)) * np.where(r.uniform(size=(M, K)) < 0.01, 20.0, 1.0)
    xb = _bf16(x)
    # codes and per-block scales drawn directly: neighbouring blocks differ by up to 2^8
    wc = r.integers(0, 256, (N, K)).astype(np.uint8)
    wc[(wc & 127) == 127] = 0
    ws = (2.0 ** r.uniform(-12, -4, (-(-N // 128), -(-K // 128)))).astype(np.float32)
    bias = _bf16(r.standard_normal(N)) if with_bias else None
    codes, scales = _quant_act(L, xb)
    xv = R.fp8_values(host(codes), host(scales)[:, :M].T, 1)
    wv = R.fp8_values(wc, ws, 128)
    need = L.fp4_linear_fp8_b128_workspace_size(M, N, K)
    work = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bd = None if bias is None else dev_bf16(bias)
    L.fp4_linear_fp8_b128(dev_bf16(xb), dev(wc), dev(ws), bd, out, M, N, K, work)
    assert L.fp4_get_device_status() == 0
    got = bf16_bits_host(out)
    _check(got, xv, wv, bias, -(-K // 128))
    # the two calls apart, on another stream, give the same bits
    out2 = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    wd, sd = dev(wc), dev(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.fp4_gemm_fp8_b128(codes, scales, wd, sd, bd, out2, M, N, K)
    torch.cuda.current_stream().wait_stream(side)
    assert np.array_equal(bf16_bits_host(out2), got)


@pytest.mark.parametrize("M", [4, 300])
def test_one_hot_rows_pick_weights_exactly(L, M):
    """A row with a single 1 (scale 1/448, code 448) returns one weight column."""
    import torch

    N, K = 264, 400
    r = np.random.default_rng(3)
    wc = r.integers(0, 255, (N, K)).astype(np.uint8)
    wc[(wc & 127) == 127] = 0
    ws = (2.0 ** r.integers(-6, 6, (3, 4))).astype(np.float32)
    x = np.zeros((M, K))
    col = r.integers(0, K, M)
    x[np.arange(M), col] = 1.0
    work = torch.zeros(L.fp4_linear_fp8_b128_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    L.fp4_linear_fp8_b128(dev_bf16(_bf16(x)), dev(wc), dev(ws), None, out, M, N, K, work)
    want = R.fp8_values(wc, ws, 128)[:, col].T
    got = bf16_bits_to_f64(bf16_bits_host(out))
    # code 448 times fp32(1/448) is within 2^-23 of one, and E4M3 times a power of two is a
    # bf16 value: the rounding returns it
    assert np.array_equal(got, want)


def test_nan_blocks_stay_in_their_rows_and_columns(L):
    import torch

    M, N, K = 40, 264, 272
    r = np.random.default_rng(9)
    x = r.standard_normal((M, K))
    x[11, 200] = np.inf
    wc = r.integers(0, 120, (N, K)).astype(np.uint8)
    ws = np.full((3, 3), 0.01, np.float32)
    ws[1, 2] = np.nan
    work = torch.zeros(L.fp4_linear_fp8_b128_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    L.fp4_linear_fp8_b128(dev_bf16(_bf16(x)), dev(wc), dev(ws), None, out, M, N, K, work)
    nan = np.isnan(bf16_bits_to_f64(bf16_bits_host(out)))
    want = np.zeros((M, N), bool)
    want[11] = True
    want[:, 128:256] = True
    assert np.array_equal(nan, want)


def test_small_workspace_is_refused(L):
    import torch

    need = L.fp4_linear_fp8_b128_workspace_size(8, 128, 128)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    t = torch.zeros(8 * 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(128, 128, dtype=torch.uint8, device="cuda")
    s = torch.ones(1, 1, device="cuda")
    with pytest.raises(L.Fp4Error) as err:
        L.fp4_linear_fp8_b128(t, w, s, None, t, 8, 128, 128, work, workspace_bytes=need - 1)
    assert err.value.status == L.FP4_ERR_INVALID_ARG


def test_two_calls_give_the_same_bits(L):
    import torch

    M, N, K = 64, 2048, 8192          # split over a cluster
    x = torch.randn(M, K, device="cuda").bfloat16()
    w = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda")
    s = torch.full((N // 128, K // 128), 0.01, device="cuda")
    work = torch.zeros(L.fp4_linear_fp8_b128_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    a, b = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.fp4_linear_fp8_b128(x, w, s, None, a, M, N, K, work)
    L.fp4_linear_fp8_b128(x, w, s, None, b, M, N, K, work)
    assert L.fp4_get_device_status() == 0
    assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 16, 32, 64, 128, 300])
def test_many_calls_give_the_same_bits(L, M):
    """Repeated calls back to back, a block's scales differing by powers of two
    from its neighbours': a scale read of the wrong block would show."""
    import torch

    N, K = 1536, 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda")
    x = (x * torch.exp2(torch.randint(-9, 9, (K // 128,), generator=g, device="cuda").repeat_interleave(128))).bfloat16()
    w = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.exp2(torch.randint(-9, 9, (N // 128, K // 128), generator=g, device="cuda").float())
    work = torch.zeros(L.fp4_linear_fp8_b128_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.empty((40, M, N), dtype=torch.bfloat16, device="cuda")
    for i in range(40):
        L.fp4_linear_fp8_b128(x, w, s, None, out[i], M, N, K, work)
    assert L.fp4_get_device_status() == 0
    assert all(torch.equal(out[0], out[i]) for i in range(1, 40))
    codes, scales = _quant_act(L, bf16_bits_host(x))
    _check(bf16_bits_host(out[39]), R.fp8_values(host(codes), host(scales)[:, :M].T, 1), R.fp8_values(host(w), host(s), 128),
           None, K // 128)


# clusters of 3 and 6 along K: tokens that they do not divide, blocks that they do not
@pytest.mark.parametrize("M,N,K", [(1, 5000, 1680), (5, 5128, 1536), (13, 9992, 768), (16, 11008, 1040), (31, 5632, 2048),
                                   (64, 10232, 896), (57, 5120, 1552), (128, 5120, 1024), (101, 4872, 784)])
def test_clusters_that_do_not_divide(L, M, N, K):
    test_linear_matches_the_formula(L, M, N, K, True)
