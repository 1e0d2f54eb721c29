"""Waits of the 8-bit product that run out on single CTAs, whichever CTA's loads are withheld: a CTA that
exists reports it, and one that does not exist changes nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


# 3 rows take 64 x 32 tiles: four CTAs, two, one
@pytest.mark.parametrize("N,ctas", [(100, 4), (33, 2), (32, 1)])
@pytest.mark.parametrize("flags", [1, 4, 5])
def test_each_cta_reports_its_loads(N, ctas, flags):
    import combine_fp32_router_gb300 as moe
    K = 500
    a = moe.moe_quantize_rows_fp8(torch.randn(3, K, device=DEV))
    b = moe.moe_quantize_blocks_fp8(torch.randn(1, K, N, device=DEV).bfloat16())
    want, o = torch.empty(3, N, device=DEV), torch.zeros(3, N, device=DEV)
    moe.moe_gemm_fp8(*a, *b, want, K)
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    moe.moe_set_wait_timeout_ns(200_000_000)
    try:
        moe.moe_debug_set_flags(flags)
        moe.moe_gemm_fp8(*a, *b, o, K)
        got = moe.moe_gemm_fp8_get_error()
    finally:
        moe.moe_debug_set_flags(0)
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    withheld = {1: 1, 4: 2, 5: 1}[flags]  # the first CTA, or the second one alone
    assert got == (moe.MOE_ERR_TIMEOUT if withheld <= ctas else moe.MOE_OK)
    if withheld > ctas:
        assert torch.equal(o, want)
    moe.moe_gemm_fp8(*a, *b, o, K)
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    assert torch.equal(o, want)
