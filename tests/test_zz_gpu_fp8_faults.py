"""Waits of the 8-bit product that run out: an error status after the limit, a usable device, and the
right result from the next call."""
import time

import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


# the first CTA's loader and, with pairs, the second one's; shapes that run on single CTAs and pairs
@pytest.mark.parametrize("flags", [1, 4, 5])
@pytest.mark.parametrize("rows,N,K", [(3, 100, 500), (200, 400, 2000), (2048, 2560, 1024)])
def test_withheld_loads(flags, rows, N, K):
    import combine_fp32_router_gb300 as moe
    a = moe.moe_quantize_rows_fp8(torch.randn(rows, K, device=DEV))
    b = moe.moe_quantize_blocks_fp8(torch.randn(1, K, N, device=DEV).bfloat16())
    want, o = torch.empty(rows, N, device=DEV), torch.zeros(rows, N, device=DEV)
    moe.moe_gemm_fp8(*a, *b, want, K)
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    moe.moe_set_wait_timeout_ns(200_000_000)
    try:
        moe.moe_debug_set_flags(flags)
        t0 = time.time()
        moe.moe_gemm_fp8(*a, *b, o, K)
        got = moe.moe_gemm_fp8_get_error()
        took = time.time() - t0
    finally:
        moe.moe_debug_set_flags(0)
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    one_cta = N <= 128 and rows <= 128  # the second CTA may not exist
    assert got == moe.MOE_ERR_TIMEOUT or (got == moe.MOE_OK and flags == 4 and one_cta)
    assert took < 5
    moe.moe_gemm_fp8(*a, *b, o, K)
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    assert torch.equal(o, want)
