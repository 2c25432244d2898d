"""Matrix-vector products whose waits run out: the call ends, reports it, writes nothing
wrong, and the next call is right.  (The test hook leaves out the first load of the
first CTA.)"""
import numpy as np
import pytest

import _layer_ref as R
from _util import dev, lib
from test_gpu_gemv import acts, check, swizzle, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return lib()


def without_a_load(L, call):
    """The status of a call whose first load never comes."""
    import torch

    torch.cuda.synchronize()
    L.fp4_debug_set_wait_fault(2_000_000, 1)
    try:
        call()
        status = L.fp4_get_device_status()
    finally:
        L.fp4_debug_set_wait_fault(0, 0)
    assert L.fp4_get_device_status() == 0
    return status


# one stage in all, several sets a CTA, more stages than the ring has places, several launches
@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (2, 16000, 1024), (1, 4096, 8192), (7, 9000, 2080), (8, 200, 65536)])
@pytest.mark.parametrize("nv", [False, True])
def test_products(L, m, n, k, nv):
    import torch

    r = np.random.default_rng(n + k)
    codes, s, w = weight(r, n, k, nv)
    x = acts(r, m, k)
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (x.cuda(), dev(codes), dev(swizzle(s)))

    def call():
        if nv:
            L.fp4_gemv_nvfp4(*args, 1.0, None, out, m, n, k)
        else:
            L.fp4_gemv_mxfp4(*args, None, out, m, n, k)

    call()
    check(out, x, w, None)
    good = out.clone()
    out.fill_(7.0)
    assert without_a_load(L, call) == L.FP4_ERR_TIMEOUT
    assert (out[:, :32] == 7.0).all()
    untouched = out == 7.0
    assert torch.equal(out[~untouched], good[~untouched])
    call()
    assert torch.equal(out, good)


# sets of one stage or two, many rows of x a CTA; rows that no expert has among them
@pytest.mark.parametrize("rows,per,n,k", [(2000, 1, 64, 1024), (2000, 4, 40, 96), (700, 1, 130, 2048), (5, 1, 8, 32)])
def test_experts(L, rows, per, n, k):
    """Warps whose wait has run out meet the others at the barrier between two rows of x."""
    import torch

    E = 4
    r = np.random.default_rng(rows + n)
    parts = [weight(r, n, k, False) for _ in range(E)]
    w = torch.stack([dev(c) for c, _, _ in parts])
    sw = torch.stack([dev(swizzle(s)) for _, s, _ in parts])
    ids = r.integers(0, E, rows).astype(np.int32)
    ids[3:rows:7] = -1
    x = acts(r, -(-rows // per), k)
    xd, idd = x.cuda(), dev(ids)
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")

    def call():
        L.fp4_gemv_mxfp4_experts(xd, idd, E, rows, per, w, sw, None, out, n, k)

    call()
    for i in list(range(min(6, rows))) + [rows - 1]:
        if ids[i] >= 0:
            check(out[i:i + 1], x[i // per:i // per + 1], parts[ids[i]][2], None)
        else:
            assert (out[i] == 0).all()
    good = out.clone()
    out.fill_(7.0)
    assert without_a_load(L, call) == L.FP4_ERR_TIMEOUT
    assert (out[0, :32] == 7.0).all()
    untouched = out == 7.0
    assert torch.equal(out[~untouched], good[~untouched])
    call()
    assert torch.equal(out, good)
