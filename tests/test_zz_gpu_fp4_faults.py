"""Failure detection of the 4-bit kernels without a GPU fault: a loader that a test hook stops
(moe_debug_set_flags) makes bounded waits run out; the call comes back with MOE_ERR_TIMEOUT, the
context stays usable and the next call is right."""
import contextlib

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@contextlib.contextmanager
def stopped(moe, flags):
    """Loaders stopped, waits of 50 ms."""
    torch.cuda.synchronize()
    try:
        moe.moe_set_wait_timeout_ns(50_000_000)
        moe.moe_debug_set_flags(flags)
        yield
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_set_flags(0)
        moe.moe_set_wait_timeout_ns(2_000_000_000)


# single CTAs (four of them; with more stages than the ring has), CTA pairs
@pytest.mark.parametrize("rows,N,K", [(1, 128, 128), (300, 256, 5000), (4000, 4096, 3000)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("flags", [1, 4, 5])
def test_product_times_out_and_recovers(moe, rows, N, K, out_dtype, flags):
    aq, sa = moe.moe_quantize_rows_fp4(torch.randn(rows, K, generator=gen(1), device=DEV))
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(1, K, N, generator=gen(2), device=DEV).to(torch.bfloat16))
    want, out = (torch.empty(rows, N, dtype=out_dtype, device=DEV) for _ in range(2))
    moe.moe_gemm_fp4(aq, sa, bq, sb, want, K)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK
    with stopped(moe, flags):
        moe.moe_gemm_fp4(aq, sa, bq, sb, out, K)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_ERR_TIMEOUT
    moe.moe_gemm_fp4(aq, sa, bq, sb, out, K)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK
    assert torch.equal(out, want)


# tokens as columns, gathered tokens, rows that are odd numbers of 128-byte pieces; more stages than
# the ring has, one stage
@pytest.mark.parametrize("T,d,E,k,dff", [(1, 4096, 8, 4, 512), (4, 384, 16, 3, 128),
                                         (16, 2048, 8, 3, 1024), (32, 128, 4, 2, 128)])
@pytest.mark.parametrize("router", [False, True])
@pytest.mark.parametrize("flags", [1, 4, 5])
def test_few_tokens_time_out_and_recover(moe, T, d, E, k, dff, router, flags):
    x = torch.randn(T, d, generator=gen(3), device=DEV).to(torch.bfloat16)
    W = [moe.moe_quantize_weights_fp4((torch.randn(E, a, b, generator=gen(4 + i), device=DEV) /
                                       a ** 0.5).to(torch.bfloat16))
         for i, (a, b) in enumerate([(d, dff), (d, dff), (dff, d)])]
    logits = torch.randn(T, E, generator=gen(7), device=DEV)
    R = torch.randn(E, d, generator=gen(8), device=DEV) / d ** 0.5 if router else None
    ws = torch.empty(moe.moe_few_workspace_bytes(T, d, E, k, dff), dtype=torch.uint8, device=DEV)
    want, out = torch.empty_like(x), torch.empty_like(x)

    def run(o):
        moe.moe_forward_few_fp4(x, logits, R, W[0][0], W[1][0], W[2][0], W[0][1], W[1][1], W[2][1],
                                k, o, ws)
    run(want)
    assert moe.moe_get_error(ws) == moe.MOE_OK
    with stopped(moe, flags):
        run(out)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_TIMEOUT
    run(out)
    assert moe.moe_get_error(ws) == moe.MOE_OK
    assert torch.equal(out, want)
