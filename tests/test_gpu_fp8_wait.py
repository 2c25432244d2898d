"""The FP8 GEMM behind a long kernel: the limit of its bounded waits counts from
when its inputs may be read, not from when its CTAs became resident."""
import numpy as np
import pytest

from _util import dev, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


# one token (K whole and in parts), a decode batch, a prefill chunk (pairs)
@pytest.mark.parametrize("M,N,K", [(1, 25600, 2048), (1, 1024, 2048), (50, 1024, 2048), (1100, 5120, 512)])
def test_a_long_kernel_ahead_is_no_timeout(L, M, N, K):
    """Ahead of the GEMM runs attention of one CTA per key head and sequence that
    takes several milliseconds in four of its CTAs (a long context on one page);
    the rest are done at once and leave their places to the GEMM, whose waits may
    last half a millisecond."""
    import torch

    heads, batch, page, long = 8, 310, 4096, 1 << 20
    cache = L.kv_cache(*(torch.zeros((1, heads, page, w), dtype=torch.uint8, device="cuda") for w in (32, 2) * 2), page, 0)
    lens = np.ones(batch, np.int32)
    lens[0] = long - 1
    table = torch.zeros((batch, long // page), dtype=torch.int32, device="cuda")
    q = torch.randn(batch, heads, 64, device="cuda").bfloat16()
    o = torch.empty_like(q)
    ctx, cu = dev(lens), torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    assert L.fp4_kv_attention_workspace_size(batch, batch, heads, heads, 64, long, 1) == 0    # no second kernel
    a = torch.randint(0, 120, (M, K), dtype=torch.uint8, device="cuda")
    b = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda")
    sa = torch.full((K // 128, -(-M // 4) * 4), 0.01, device="cuda")
    sb = torch.full((-(-N // 128), K // 128), 0.01, device="cuda")
    want, got = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    attend = lambda: L.fp4_kv_attention(cache, q, o, table, ctx, cu, long, 1, None)  # noqa: E731
    L.fp4_gemm_fp8_b128(a, sa, b, sb, None, want, M, N, K)
    attend()
    assert L.fp4_get_device_status() == 0
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    attend()
    t[1].record()
    torch.cuda.synchronize()
    assert t[0].elapsed_time(t[1]) > 2.0
    L.fp4_debug_set_wait_fault(500_000, 0)
    try:
        attend()
        L.fp4_gemm_fp8_b128(a, sa, b, sb, None, got, M, N, K)
        assert L.fp4_get_device_status() == 0
    finally:
        L.fp4_debug_set_wait_fault(0, 0)
    assert torch.equal(got, want)
