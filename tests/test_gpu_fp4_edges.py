"""The 4-bit operators at their edges on the GPU: repeated runs, values that are not finite, wide
layers, matrices of more than 2^31 values, and what the few-token layer keeps of its activations."""
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ------------------------------------------------------------------------- product
@pytest.mark.parametrize("rows,N,K", [(4000, 4096, 640), (2049, 2048, 3000)])
def test_pairs_repeat_bit_for_bit(moe, rows, N, K):
    """Products on CTA pairs, whose waits see the peer's arrivals: twenty runs, one after the other,
    give the bits of the first."""
    aq, sa = moe.moe_quantize_rows_fp4(torch.randn(rows, K, generator=gen(1), device=DEV))
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(1, K, N, generator=gen(2), device=DEV).to(torch.bfloat16))
    outs = [torch.empty(rows, N, device=DEV) for _ in range(20)]
    for o in outs:
        moe.moe_gemm_fp4(aq, sa, bq, sb, o, K)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK
    av, bv = ref.values(aq, sa, rows, K), ref.values(bq[0], sb[0], N, K)
    bound = (K + 8) * 2.0 ** -23 * (av.abs() @ bv.abs().t())
    assert ref.within(outs[0], av @ bv.t(), bound)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_an_error_is_taken_by_one_caller(moe):
    """Callers that read the record at once: one of them gets the error, the record is clear then."""
    import threading
    aq, sa = moe.moe_quantize_rows_fp4(torch.randn(128, 128, generator=gen(3), device=DEV))
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(2, 128, 128, generator=gen(4), device=DEV).to(torch.bfloat16))
    out = torch.empty(128, 128, device=DEV)
    bad = torch.tensor([128, 1], dtype=torch.int32, device=DEV)
    n, rounds = 8, 40
    streams = [torch.cuda.Stream() for _ in range(n)]
    barrier = threading.Barrier(n + 1)
    got = [[] for _ in range(n)]

    def reader(i):
        for _ in range(rounds):
            barrier.wait()
            got[i].append(moe.moe_gemm_fp4_get_error(streams[i]))
            barrier.wait()
    threads = [threading.Thread(target=reader, args=(i,), daemon=True) for i in range(n)]
    for t in threads:
        t.start()
    for _ in range(rounds):
        moe.moe_gemm_fp4(aq, sa, bq, sb, out, 128, counts=bad)
        torch.cuda.synchronize()
        barrier.wait(60)
        barrier.wait(60)
    for t in threads:
        t.join(60)
    for r in range(rounds):
        statuses = sorted(g[r] for g in got)
        assert statuses == [moe.MOE_OK] * (n - 1) + [moe.MOE_ERR_DEVICE_BOUNDS], r
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


@pytest.mark.parametrize("counts", [[133], [133, 0, 0], [0, 133, 0], [128, 5] + [0] * 40, [5, 200, 0],
                                    [3000, 1500, 0, 0]])
def test_rows_may_end_with_the_last_segment(moe, counts):
    """Rows that stop where the last expert's do, with no padding for the experts after it that have
    none; one row fewer does not hold the segments."""
    E, N, K = len(counts), 1024, 256
    last = max(e for e in range(E) if counts[e])
    rows = sum(ref.up(c, 128) for c in counts[:last]) + counts[last]
    aq, sa = moe.moe_quantize_rows_fp4(torch.randn(rows, K, generator=gen(60), device=DEV))
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(E, K, N, generator=gen(61), device=DEV).to(torch.bfloat16))
    on_device = torch.tensor(counts, dtype=torch.int32, device=DEV)
    out = torch.full((rows, N), 7.0, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq, sb, out, K, counts=on_device)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK
    at = 0
    for e, c in enumerate(counts):
        if c:
            alone = torch.empty(c, N, device=DEV)
            q, s = moe.moe_quantize_rows_fp4(
                moe.moe_dequantize_rows_fp4(aq, sa, K, torch.float32)[at:at + c])
            moe.moe_gemm_fp4(q, s, bq[e], sb[e], alone, K)
            assert torch.equal(out[at:at + c], alone)
            assert bool((out[at + c:at + ref.up(c, 128)] == 7.0).all())
        at += ref.up(c, 128)
    moe.moe_gemm_fp4(aq, sa, bq, sb, out[:rows - 1], K, counts=on_device)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_ERR_DEVICE_BOUNDS


# ------------------------------------------------------------------------- few tokens
def weights(moe, d, E, dff, seed):
    return [moe.moe_quantize_weights_fp4((torch.randn(E, a, b, generator=gen(seed + i), device=DEV) /
                                          a ** 0.5).to(torch.bfloat16))
            for i, (a, b) in enumerate([(d, dff), (d, dff), (dff, d)])]


def run_few(moe, x, logits, router, W, k):
    T, d = x.shape
    E, dff = W[0][0].shape[:2]
    ws = torch.full((moe.moe_few_workspace_bytes(T, d, E, k, dff),), 255, dtype=torch.uint8,
                    device=DEV)
    out = torch.full((T, d), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_forward_few_fp4(x, logits, router, W[0][0], W[1][0], W[2][0], W[0][1], W[1][1],
                            W[2][1], k, out, ws)
    assert moe.moe_get_error(ws) == moe.MOE_OK
    return out


def dense(W, rows, cols):
    return torch.stack([ref.values(q, s, rows, cols) for q, s in zip(*W)])


# the widths of large layers, up to the largest; sums of more than eight K ranges (d > 8192); experts
# with more than eight tokens
@pytest.mark.parametrize("T,d,E,k,dff", [
    (1, 7168, 4, 2, 256), (8, 4096, 5, 3, 384), (32, 7168, 8, 2, 128), (5, 8320, 2, 2, 128),
    (16, 16384, 3, 2, 128), (2, 65536, 2, 1, 128), (3, 128, 2, 1, 65536), (9, 384, 3, 2, 8320)])
def test_few_wide_layers(moe, T, d, E, k, dff):
    x = torch.randn(T, d, generator=gen(20), device=DEV).to(torch.bfloat16)
    W = weights(moe, d, E, dff, 21)
    router = torch.randn(E, d, generator=gen(25), device=DEV) / d ** 0.5
    logits = torch.full((T, E), float("nan"), device=DEV)
    out = run_few(moe, x, logits, router, W, k)
    want = x.double() @ router.double().t()
    u = (d + 8) * 2.0 ** -24 * (x.double().abs() @ router.double().abs().t())
    assert bool(((logits.double() - want).abs() <= u).all())
    want, bound = ref.few_in_terms(x, logits, dense(W[0], dff, d), dense(W[1], dff, d),
                                   dense(W[2], d, dff), k)
    assert ref.within(out, want, bound)
