"""MXFP4 quantisation, the product of quantised matrices, and the few-token layer on the GPU
against 64-bit arithmetic (tests/fp4_reference.py)."""
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


def special_rows(cols, dtype):
    """Rows of zeros, ties, the type's extremes, subnormals and mixed magnitudes."""
    fi = torch.finfo(dtype)
    ties = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 7.0, 7.9])
    rows = [torch.zeros(cols), ties.repeat(cols // 12 + 1)[:cols],
            torch.full((cols,), fi.max), torch.full((cols,), fi.tiny),
            torch.full((cols,), fi.smallest_normal / 4), -torch.ones(cols),
            torch.logspace(-30, 4, cols).clamp(max=fi.max)]
    z = torch.zeros(cols)
    z[0] = -0.0
    rows.append(z)
    return torch.stack(rows).to(dtype).to(DEV)


# ------------------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 31, 0), (3, 32, 5), (5, 33, 0),
                                           (130, 127, 1), (127, 128, 0), (129, 1000, 24),
                                           (8, 7168, 0), (257, 1025, 3), (2, 4100, 4)])
def test_quantize_rows_is_exact(moe, dtype, rows, cols, pad):
    x = (torch.randn(rows, cols + pad, generator=gen(1), device=DEV) *
         torch.exp2(torch.randint(-6, 6, (rows, 1), generator=gen(2), device=DEV))).to(dtype)
    x = x[:, pad:] if pad % 2 else x[:, :cols]   # an odd first column: unaligned rows
    q, s = moe.moe_quantize_rows_fp4(x)
    want = ref.quantized(x)
    assert torch.equal(ref.values(q, s, rows, cols), want)
    # the rest of a row is zero codes, the rows that the last tile adds have scale bytes 0
    assert int(q.view(rows, -1)[:, (cols + 1) // 2:].max() if cols <= q.shape[1] * 2 - 2 else 0) == 0
    kt = q.shape[1] // 64
    tiles = s.view(-1, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kt * 4)
    assert int(tiles[rows:].sum()) == 0
    back = moe.moe_dequantize_rows_fp4(q, s, cols, torch.float32)
    assert torch.equal(back.double(), want)
    assert torch.equal(moe.moe_dequantize_rows_fp4(q, s, cols, torch.bfloat16).double(), want)
    assert torch.equal(moe.moe_dequantize_rows_fp4(q, s, cols, torch.float16), want.half())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", [96, 101])
def test_quantize_special_values(moe, dtype, cols):
    x = special_rows(cols, dtype)
    q, s = moe.moe_quantize_rows_fp4(x)
    assert torch.equal(ref.values(q, s, x.shape[0], cols), ref.quantized(x))


def test_non_finite_blocks_are_nan_and_alone(moe):
    x = torch.randn(4, 256, generator=gen(3), device=DEV)
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2, 255] = -float("inf")
    q, s = moe.moe_quantize_rows_fp4(x)
    want = ref.quantized(x)
    back = moe.moe_dequantize_rows_fp4(q, s, 256, torch.float32).double()
    assert int(torch.isnan(back).sum()) == 96
    assert torch.equal(torch.nan_to_num(back, 99.0), torch.nan_to_num(want, 99.0))


@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (2, 32, 8), (3, 100, 65), (2, 257, 130),
                                   (1, 300, 63), (4, 512, 128), (2, 128, 264)])
def test_quantize_weights_is_exact(moe, E, K, N):
    W = (torch.randn(E, K, N, generator=gen(4), device=DEV) / 8).to(torch.bfloat16)
    W[0, :, 0] = 0
    if K > 40 and N > 3:
        W[0, 33, 3] = float("inf")
    q, s = moe.moe_quantize_weights_fp4(W)
    for e in range(E):
        want = ref.quantized(W[e].t().contiguous())
        got = ref.values(q[e], s[e], N, K)
        assert torch.equal(torch.nan_to_num(got, 99.0), torch.nan_to_num(want, 99.0))
    back = moe.moe_dequantize_rows_fp4(q, s, K, torch.float32)
    for e in range(E):
        assert torch.equal(torch.nan_to_num(back[e].double(), 99.0),
                           torch.nan_to_num(ref.values(q[e], s[e], N, K), 99.0))


def test_quantize_no_rows(moe):
    q, s = moe.moe_quantize_rows_fp4(torch.empty(0, 64, device=DEV))
    assert q.shape == (0, 64) and s.numel() == 0
    assert moe.moe_dequantize_rows_fp4(q, s, 64).shape == (0, 64)


# ------------------------------------------------------------------------- product
def gemm_bound(a, b):
    """fp32 accumulation in any order, each addition off by at most 2^-23 of the partial sum's
    bound."""
    return (a.shape[1] + 8) * 2.0 ** -23 * (a.abs() @ b.abs().t())


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 1), (1, 128, 128), (3, 129, 257), (16, 64, 384),
                                      (17, 200, 100), (64, 130, 640), (65, 96, 512),
                                      (128, 256, 1000), (129, 33, 129), (192, 128, 256),
                                      (193, 257, 1537), (384, 128, 130), (500, 512, 3001)])
def test_gemm_dense(moe, rows, N, K, out_dtype):
    a = torch.randn(rows, K, generator=gen(5), device=DEV) * \
        torch.exp2(torch.randint(-9, 9, (rows, K), generator=gen(6), device=DEV))
    b = (torch.randn(1, K, N, generator=gen(7), device=DEV) / 16).to(torch.bfloat16)
    aq, sa = moe.moe_quantize_rows_fp4(a)
    bq, sb = moe.moe_quantize_weights_fp4(b)
    out = torch.full((rows, N), 7.0, dtype=out_dtype, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq[0], sb, out, K)
    av, bv = ref.values(aq, sa, rows, K), ref.values(bq[0], sb[0], N, K)
    want = av @ bv.t()
    assert ref.within(out, want, gemm_bound(av, bv))
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


@pytest.mark.parametrize("counts", [[1], [0, 5, 0], [128, 129, 127, 0, 1], [0, 0, 0],
                                    [300, 0, 192, 193, 384, 64, 65], [3] * 40])
@pytest.mark.parametrize("N,K", [(96, 160), (300, 512)])
def test_gemm_grouped(moe, counts, N, K):
    E, rows = len(counts), sum(ref.up(c, 128) for c in counts) + 128
    a = torch.randn(rows, K, generator=gen(8), device=DEV)
    b = torch.randn(E, K, N, generator=gen(9), device=DEV).to(torch.bfloat16)
    aq, sa = moe.moe_quantize_rows_fp4(a)
    bq, sb = moe.moe_quantize_weights_fp4(b)
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq, sb, out, K,
                     counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
    av = ref.values(aq, sa, rows, K)
    at, kept = 0, torch.ones(rows, dtype=torch.bool, device=DEV)
    for e, c in enumerate(counts):
        if c:
            bv = ref.values(bq[e], sb[e], N, K)
            want = av[at:at + c] @ bv.t()
            assert ref.within(out[at:at + c], want, gemm_bound(av[at:at + c], bv))
        kept[at:at + c] = False
        at += ref.up(c, 128)
    assert bool((out[kept] == 7.0).all())
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


def test_gemm_rows_do_not_depend_on_the_batch(moe):
    K, N = 1500, 300
    a = torch.randn(400, K, generator=gen(10), device=DEV)
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(1, K, N, generator=gen(11), device=DEV).to(torch.bfloat16))

    def product(rows):
        q, s = moe.moe_quantize_rows_fp4(rows)
        o = torch.empty(rows.shape[0], N, device=DEV)
        moe.moe_gemm_fp4(q, s, bq, sb, o, K)
        return o
    whole = product(a)
    for n in (1, 2, 17, 100, 193, 399):
        assert torch.equal(product(a[:n]), whole[:n])
    assert torch.equal(product(a.flip(0)).flip(0), whole)


def test_gemm_tile_shapes_give_the_same_bits(moe):
    """Many rows run on CTA pairs, a hundred of them alone on single CTAs, ten on single CTAs with
    fewer weight rows each."""
    rows, K, N = 4000, 600, 4096
    a = torch.randn(rows, K, generator=gen(110), device=DEV)
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(1, K, N, generator=gen(111), device=DEV).to(torch.bfloat16))

    def product(x):
        q, s = moe.moe_quantize_rows_fp4(x)
        o = torch.empty(x.shape[0], N, device=DEV)
        moe.moe_gemm_fp4(q, s, bq, sb, o, K)
        return o
    whole = product(a)
    for first, n in ((0, 100), (1234, 100), (3990, 10), (2000, 1)):
        assert torch.equal(product(a[first:first + n].contiguous()), whole[first:first + n])
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


def test_gemm_grouped_on_pairs(moe):
    counts, N, K = [2000, 0, 1500, 193, 64, 3000, 1, 700], 2048, 384
    E, rows = len(counts), sum(ref.up(c, 128) for c in counts)
    a = torch.randn(rows, K, generator=gen(112), device=DEV)
    b = torch.randn(E, K, N, generator=gen(113), device=DEV).to(torch.bfloat16)
    aq, sa = moe.moe_quantize_rows_fp4(a)
    bq, sb = moe.moe_quantize_weights_fp4(b)
    out = torch.full((rows, N), 7.0, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq, sb, out, K,
                     counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
    av = ref.values(aq, sa, rows, K)
    at = 0
    for e, c in enumerate(counts):
        bv = ref.values(bq[e], sb[e], N, K)
        assert ref.within(out[at:at + c], av[at:at + c] @ bv.t(), gemm_bound(av[at:at + c], bv))
        assert bool((out[at + c:at + ref.up(c, 128)] == 7.0).all())
        at += ref.up(c, 128)
    assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK


def test_gemm_nan_scales_reach_their_rows_and_columns_only(moe):
    a = torch.randn(200, 256, generator=gen(12), device=DEV)
    a[150, 70] = float("inf")
    b = torch.randn(1, 256, 140, generator=gen(13), device=DEV).to(torch.bfloat16)
    b[0, 3, 135] = float("nan")
    aq, sa = moe.moe_quantize_rows_fp4(a)
    bq, sb = moe.moe_quantize_weights_fp4(b)
    out = torch.empty(200, 140, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq, sb, out, 256)
    nan = torch.zeros(200, 140, dtype=torch.bool, device=DEV)
    nan[150] = True
    nan[:, 135] = True
    assert torch.equal(torch.isnan(out), nan)


def test_gemm_counts_that_do_not_fit(moe):
    K, N = 128, 128
    aq, sa = moe.moe_quantize_rows_fp4(torch.randn(256, K, generator=gen(14), device=DEV))
    bq, sb = moe.moe_quantize_weights_fp4(
        torch.randn(2, K, N, generator=gen(15), device=DEV).to(torch.bfloat16))
    for counts in ([129, 1], [-1, 3], [0, 257]):
        out = torch.full((256, N), 7.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_gemm_fp4(aq, sa, bq, sb, out, K,
                         counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
        assert bool((out == 7.0).all())
        assert moe.moe_gemm_fp4_get_error() == moe.MOE_ERR_DEVICE_BOUNDS
        assert moe.moe_gemm_fp4_get_error() == moe.MOE_OK   # cleared by the read
    out = torch.full((256, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq, sb, out, K,
                     counts=torch.tensor([128, 128], dtype=torch.int32, device=DEV))
    assert bool((out != 7.0).any()) and moe.moe_gemm_fp4_get_error() == moe.MOE_OK


def test_gemm_on_another_stream(moe):
    a = torch.randn(64, 512, generator=gen(16), device=DEV)
    b = torch.randn(1, 512, 256, generator=gen(17), device=DEV).to(torch.bfloat16)
    bq, sb = moe.moe_quantize_weights_fp4(b)
    aq, sa = moe.moe_quantize_rows_fp4(a)
    base = torch.empty(64, 256, device=DEV)
    moe.moe_gemm_fp4(aq, sa, bq, sb, base, 512)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros(64, 256, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    q2, s2 = torch.empty_like(aq), torch.empty_like(sa)
    moe.moe_quantize_rows_fp4(a, q2, s2, stream=s)
    moe.moe_gemm_fp4(q2, s2, bq, sb, out, 512, stream=s)
    s.synchronize()
    assert torch.equal(out, base)


def test_new_outputs_on_another_stream(moe):
    x = torch.randn(300, 700, generator=gen(18), device=DEV)
    W = torch.randn(2, 300, 96, generator=gen(19), device=DEV).to(torch.bfloat16)
    q0, s0 = moe.moe_quantize_rows_fp4(x)
    w0, ws0 = moe.moe_quantize_weights_fp4(W)
    v0 = moe.moe_dequantize_rows_fp4(q0, s0, 700, torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q1, s1 = moe.moe_quantize_rows_fp4(x, stream=s)
    w1, ws1 = moe.moe_quantize_weights_fp4(W, stream=s)
    v1 = moe.moe_dequantize_rows_fp4(q1, s1, 700, torch.float32, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in ((q0, q1), (s0, s1), (w0, w1), (ws0, ws1), (v0, v1)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------- few tokens
def layer(moe, T, d, E, k, dff, seed, spread=0):
    x = torch.randn(T, d, generator=gen(seed), device=DEV).to(torch.bfloat16)
    if spread:
        x = (x.float() * torch.exp2(torch.randint(-spread, spread, (T, d), generator=gen(seed + 1),
                                                  device=DEV))).to(torch.bfloat16)
    W = [(torch.randn(E, a, b, generator=gen(seed + 2 + i), device=DEV) / a ** 0.5).to(torch.bfloat16)
         for i, (a, b) in enumerate([(d, dff), (d, dff), (dff, d)])]
    return x, [moe.moe_quantize_weights_fp4(w) for w in W]


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


def dense(W, E, rows, cols):
    return torch.stack([ref.values(W[0][e], W[1][e], rows, cols) for e in range(E)])


@pytest.mark.parametrize("T,d,E,k,dff,spread", [
    (1, 128, 1, 1, 128, 0), (1, 256, 4, 2, 384, 0), (2, 384, 8, 8, 128, 3), (5, 512, 16, 3, 256, 0),
    (8, 128, 8, 2, 256, 6), (9, 1152, 5, 4, 128, 0), (32, 256, 2, 2, 128, 0), (31, 640, 40, 16, 256, 0),
    (17, 1024, 300, 5, 128, 0), (32, 2048, 3, 1, 1152, 2), (3, 128, 1024, 16, 128, 0)])
def test_few_against_64_bits(moe, T, d, E, k, dff, spread):
    x, W = layer(moe, T, d, E, k, dff, 20, spread)
    logits = torch.randn(T, E, generator=gen(30), device=DEV)
    out = run_few(moe, x, logits, None, W, k)
    want, bound = ref.few(x, logits, dense(W[0], E, dff, d), dense(W[1], E, dff, d),
                          dense(W[2], E, d, dff), k)
    assert ref.within(out, want, bound)


@pytest.mark.parametrize("T", [1, 4, 7, 32])
@pytest.mark.parametrize("d,E", [(128, 7), (1152, 33), (2176, 256)])
def test_few_router_logits(moe, T, d, E):
    k, dff = 3, 128
    x, W = layer(moe, T, d, E, k, dff, 40)
    router = torch.randn(E, d, generator=gen(41), device=DEV) / d ** 0.5
    logits = torch.full((T, E), float("nan"), device=DEV)
    out = run_few(moe, x, logits, router, W, k)
    want = x.double() @ router.double().t()
    bound = (d + 8) * 2.0 ** -24 * (x.double().abs() @ router.double().abs().t())
    assert bool(((logits.double() - want).abs() <= bound).all())
    # the layer that follows is the one that reads these logits
    assert torch.equal(out, run_few(moe, x, logits.clone(), None, W, k))


def test_few_tokens_do_not_depend_on_the_batch(moe):
    T, d, E, k, dff = 32, 640, 12, 4, 256
    x, W = layer(moe, T, d, E, k, dff, 50)
    router = torch.randn(E, d, generator=gen(51), device=DEV) / d ** 0.5
    logits = torch.empty(T, E, device=DEV)
    whole = run_few(moe, x, logits, router, W, k)
    for n in (1, 2, 3, 8, 9, 20):
        part_logits = torch.empty(n, E, device=DEV)
        assert torch.equal(run_few(moe, x[:n].contiguous(), part_logits, router, W, k), whole[:n])
        assert torch.equal(part_logits, logits[:n])
    turned = run_few(moe, x.flip(0).contiguous(), torch.empty(T, E, device=DEV), router, W, k)
    assert torch.equal(turned.flip(0), whole)
    for _ in range(5):
        assert torch.equal(run_few(moe, x, logits, router, W, k), whole)


def test_few_ties_go_to_the_lower_expert(moe):
    T, d, E, k, dff = 3, 128, 6, 2, 128
    x, W = layer(moe, T, d, E, k, dff, 60)
    logits = torch.zeros(T, E, device=DEV)
    logits[1, 4] = -0.0
    logits[2, 5] = 1.0
    out = run_few(moe, x, logits, None, W, k)
    want, bound = ref.few(x, logits, dense(W[0], E, dff, d), dense(W[1], E, dff, d),
                          dense(W[2], E, d, dff), k)
    assert ref.within(out, want, bound)


def test_few_extreme_magnitudes(moe):
    """Tokens of zeros, of very large and very small values beside ordinary ones."""
    T, d, E, k, dff = 4, 256, 4, 2, 128
    x, W = layer(moe, T, d, E, k, dff, 70)
    x[0] = 0
    x[1] = x[1] * 1e15
    x[2] = x[2] * 1e-18
    logits = torch.randn(T, E, generator=gen(71), device=DEV)
    out = run_few(moe, x, logits, None, W, k)
    want, bound = ref.few(x, logits, dense(W[0], E, dff, d), dense(W[1], E, dff, d),
                          dense(W[2], E, d, dff), k)
    assert bool((out[0] == 0).all())
    # fp32's smallest normal number bounds what a product of tiny factors can lose
    assert ref.within(out, want, bound + 2.0 ** -126)


def test_few_nan_weights_poison_their_expert_only(moe):
    T, d, E, k, dff = 2, 256, 2, 1, 128
    x, W = layer(moe, T, d, E, k, dff, 80)
    W2 = (torch.randn(E, dff, d, generator=gen(81), device=DEV)).to(torch.bfloat16)
    W2[1, 3, 5] = float("nan")
    W[2] = moe.moe_quantize_weights_fp4(W2)
    logits = torch.tensor([[1.0, 0.0], [0.0, 1.0]], device=DEV)
    out = run_few(moe, x, logits, None, W, k)
    nan = torch.zeros(T, d, dtype=torch.bool, device=DEV)
    nan[1, 5] = True
    assert torch.equal(torch.isnan(out), nan)


def test_few_no_tokens(moe):
    x, W = layer(moe, 1, 128, 2, 1, 128, 90)
    out = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    moe.moe_forward_few_fp4(x[:0], torch.empty(0, 2, device=DEV), None, W[0][0], W[1][0], W[2][0],
                            W[0][1], W[1][1], W[2][1], 1, out,
                            torch.empty(256, dtype=torch.uint8, device=DEV))


def test_few_in_a_graph(moe):
    """Both launches captured and replayed on new tokens."""
    T, d, E, k, dff = 4, 256, 8, 2, 128
    x, W = layer(moe, T, d, E, k, dff, 100)
    router = torch.randn(E, d, generator=gen(101), device=DEV) / d ** 0.5
    logits, out = torch.empty(T, E, device=DEV), torch.empty_like(x)
    ws = torch.empty(moe.moe_few_workspace_bytes(T, d, E, k, dff), dtype=torch.uint8, device=DEV)
    args = (x, logits, router, W[0][0], W[1][0], W[2][0], W[0][1], W[1][1], W[2][1], k, out, ws)
    moe.moe_forward_few_fp4(*args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_forward_few_fp4(*args)
    x2 = torch.randn(T, d, generator=gen(102), device=DEV).to(torch.bfloat16)
    want = run_few(moe, x2, torch.empty(T, E, device=DEV), router, W, k)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------------- together
@pytest.mark.parametrize("T,d,E,k,dff", [(300, 256, 8, 2, 256), (64, 384, 5, 3, 128)])
def test_example_paths_agree(T, d, E, k, dff):
    """The example's prompt path and few-token path on one set of quantised weights.  The few-token
    path differs from the bf16 layer on the dequantised weights by the bf16 roundings of h and of
    the expert rows there (2^-9 each, rms); 4-bit weights alone are 8 to 16 percent off, and 4-bit
    rows and h add up to as much each."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp4_experts.py")
    spec = importlib.util.spec_from_file_location("fp4_experts", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    _, _, prompt, step, exact = ex.run(T, d, E, k, dff)
    assert exact < 2.0 ** -7
    assert 0.02 < step < 0.3
    assert 0.02 < prompt < 0.5
