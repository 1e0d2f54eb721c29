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


def test_product_of_more_than_2_31_outputs(moe):
    """Output places past 2^31 values, in 16-byte and in single stores; each row as alone."""
    rows, K = (1 << 20) + 77, 100
    x = torch.randn(rows, K, generator=gen(5), device=DEV, dtype=torch.bfloat16)
    for N, dtype in ((2056, torch.bfloat16), (2051, torch.float32)):
        assert rows * N > 1 << 31
        bq, sb = moe.moe_quantize_weights_fp4(
            torch.randn(1, K, N, generator=gen(6), device=DEV).to(torch.bfloat16))
        out = torch.empty(rows, N, dtype=dtype, device=DEV)
        moe.moe_gemm_fp4(*moe.moe_quantize_rows_fp4(x), bq, sb, out, K)
        for r in (0, (1 << 31) // N - 64, rows - 130):
            part = torch.empty(130, N, dtype=dtype, device=DEV)
            moe.moe_gemm_fp4(*moe.moe_quantize_rows_fp4(x[r:r + 130].contiguous()), bq, sb, part, K)
            assert torch.equal(out[r:r + 130], part)
        del out
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


def test_product_with_more_than_2_31_bytes_of_weights(moe):
    E, N, K = 512, 4096, 2080
    bq = torch.randint(0, 256, (E, N, moe.moe_fp4_row_bytes(K)), generator=gen(7), device=DEV,
                       dtype=torch.uint8)
    sb = torch.randint(120, 130, (E, moe.moe_fp4_scale_bytes(N, K)), generator=gen(8), device=DEV,
                       dtype=torch.uint8)
    assert bq.numel() > 1 << 31
    aq, sa = moe.moe_quantize_rows_fp4(torch.randn(133, K, generator=gen(9), device=DEV))
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    for e in (0, E - 1):
        counts.zero_()
        counts[e] = 133
        out, alone = (torch.empty(133, N, device=DEV) for _ in range(2))
        moe.moe_gemm_fp4(aq, sa, bq, sb, out, K, counts=counts)
        moe.moe_gemm_fp4(aq, sa, bq[e], sb[e], alone, K)
        assert torch.equal(out, alone)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


# ------------------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pad", [0, 1])
def test_blocks_that_are_not_finite(moe, dtype, pad):
    """Infinities and NaN (of either sign) make their block NaN and leave the others alone, in
    aligned rows and in others."""
    x = torch.randn(6, 256 + pad, generator=gen(10), device=DEV).to(dtype)[:, pad:]
    for r, c, v in ((0, 5, "inf"), (1, 40, "nan"), (2, 255, "-inf"), (4, 128, "-nan"), (4, 0, "inf")):
        x[r, c] = float(v) if v != "-nan" else torch.tensor(float("nan")).neg()
    q, s = moe.moe_quantize_rows_fp4(x)
    want = ref.quantized(x)
    got = ref.values(q, s, 6, 256)
    assert int(torch.isnan(got).sum()) == 5 * 32
    assert torch.equal(torch.nan_to_num(got, 99.0), torch.nan_to_num(want, 99.0))
    for to in (torch.bfloat16, torch.float16, torch.float32):
        back = moe.moe_dequantize_rows_fp4(q, s, 256, to)
        assert torch.equal(torch.isnan(back), torch.isnan(got))
        assert torch.equal(torch.nan_to_num(back.double(), 99.0), torch.nan_to_num(got, 99.0))


@pytest.mark.parametrize("cols", [1056, 1057])
def test_quantize_more_than_2_31_values(moe, cols):
    rows = (1 << 21) + 77
    assert rows * cols > 1 << 31
    x = torch.randn(rows, cols, generator=gen(11), device=DEV, dtype=torch.bfloat16)
    q, s = moe.moe_quantize_rows_fp4(x)
    back = moe.moe_dequantize_rows_fp4(q, s, cols)
    kt = q.shape[1] // 64
    for r in (0, (1 << 31) // cols // 128 * 128, (rows - 130) // 128 * 128):
        n = min(256, rows - r)
        part = ref.values(q[r:r + n], s[r // 128 * kt * 512:], n, cols)
        assert torch.equal(part, ref.quantized(x[r:r + n]))
        assert torch.equal(back[r:r + n].double(), part)


def test_quantize_more_than_2_31_weights(moe):
    E, K, N = 512, 1056, 4104
    W = torch.randn(E, K, N, generator=gen(12), device=DEV, dtype=torch.bfloat16)
    assert W.numel() > 1 << 31
    q, s = moe.moe_quantize_weights_fp4(W)
    back = moe.moe_dequantize_rows_fp4(q, s, K)
    for e in (0, E - 1):
        want = ref.quantized(W[e].t().contiguous())
        assert torch.equal(ref.values(q[e], s[e], N, K), want)
        assert torch.equal(back[e].double(), want)


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


@pytest.mark.parametrize("T", [8, 32])
def test_few_keeps_six_terms_of_its_activations(moe, T):
    """A layer that hands single values of x through: out[t, n] = silu(x[t, 0]) x[t, c] with one large
    value in each block of x, so what the terms leave of x and of h shows in the small ones, above
    bf16's rounding.  Its root mean square has to be what six terms leave; five for either would leave
    more than twice that (checked here on the reference)."""
    d, dff, E = 256, 128, 2
    x = torch.randn(T, d, generator=gen(30), device=DEV) * 2.0 ** -8
    x[:, ::32] = 32 * (1 + torch.rand(T, 8, generator=gen(31), device=DEV))
    x = x.to(torch.bfloat16)
    W1, W3 = (torch.zeros(E, d, dff, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    W2 = torch.zeros(E, dff, d, dtype=torch.bfloat16, device=DEV)
    n = torch.arange(dff, device=DEV)
    W1[:, 0] = 1
    W3[0, n, n] = 1
    W3[1, 128 + n, n] = 1
    W2[:, n, n] = 1
    logits = torch.zeros(T, E, device=DEV)
    expert = torch.arange(T, device=DEV) % E
    logits[torch.arange(T, device=DEV), expert] = 1.0
    out = run_few(moe, x, logits, None, [moe.moe_quantize_weights_fp4(w) for w in (W1, W3, W2)], 1)

    def layer(v, of_x, of_h):
        v = ref.in_terms(v, of_x) if of_x else v.double()
        h = v[:, :1] * torch.sigmoid(v[:, :1]) * v.view(T, 2, dff)[torch.arange(T, device=DEV), expert]
        return ref.in_terms(h, of_h) if of_h else h
    true = layer(x, 0, 0)
    small = torch.arange(dff, device=DEV) % 32 != 0

    def rms(v):  # of the small values, relative to the largest of their block of h
        r = ((v.double() - true) / ref.block_max(true))[:, small]
        return float((r * r).mean().sqrt())
    six = rms(layer(x, 6, 6).float().to(torch.bfloat16))
    limit = 1.5 * six
    assert rms(layer(x, 5, 6).float().to(torch.bfloat16)) > limit
    assert rms(layer(x, 6, 5).float().to(torch.bfloat16)) > limit
    assert rms(out[:, :dff]) <= limit
    worst = ((out[:, :dff].double() - true).abs() / ref.block_max(true)).max()
    assert float(worst) <= 2 * ref.LEFT + 2.0 ** -8
    assert bool((out[:, dff:] == 0).all())


@pytest.mark.parametrize("T", [5, 20])
def test_few_values_that_are_not_finite_stay_with_their_token(moe, T):
    """An infinity or a NaN in x, and an h that overflows, make their token's output NaN; the others
    come out as without them."""
    d, E, k, dff = 384, 4, 2, 256
    x = torch.randn(T, d, generator=gen(40), device=DEV).to(torch.bfloat16)
    W = weights(moe, d, E, dff, 41)
    logits = torch.randn(T, E, generator=gen(45), device=DEV)
    want = run_few(moe, x, logits, None, W, k)
    y = x.clone()
    y[0, 5] = float("inf")
    y[2, 200] = float("nan")
    y[3] *= 1e30        # a and b of 1e30, products past fp32
    out = run_few(moe, y, logits, None, W, k)
    lost = torch.zeros(T, dtype=torch.bool, device=DEV)
    lost[[0, 2, 3]] = True
    assert bool(torch.isnan(out[lost]).all())
    assert torch.equal(out[~lost], want[~lost])


def test_few_with_more_than_2_31_bytes_of_weights(moe):
    E, d, dff = 1024, 2304, 2048
    g = gen(50)

    def codes(n, K):
        q = torch.randint(0, 256, (E, n, moe.moe_fp4_row_bytes(K)), generator=g, device=DEV,
                          dtype=torch.uint8)
        s = torch.randint(114, 118, (E, moe.moe_fp4_scale_bytes(n, K)), generator=g, device=DEV,
                          dtype=torch.uint8)
        return q, s
    W = [codes(dff, d), codes(dff, d), codes(d, dff)]
    assert W[0][0].numel() > 1 << 31
    for T in (2, 12):
        x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
        logits = torch.zeros(T, E, device=DEV)
        logits[:, E - 1] = 20.0
        logits[:, 700] = 19.0
        out = run_few(moe, x, logits, None, W, 2)
        two = [(q[[E - 1, 700]].contiguous(), s[[E - 1, 700]].contiguous()) for q, s in W]
        alone = run_few(moe, x, torch.tensor([[20.0, 19.0]], device=DEV).repeat(T, 1), None, two, 2)
        assert bool((alone != 0).any()) and torch.equal(out, alone)
