"""8-bit rows and weights with a scale per 128 values and their product, on the GPU.

Quantisation of rows and blocks is a function of fp32 operations: equal.  SwiGLU's fp32 value is
within (6 + |a|) 2^-23 of the exact one.  A product's block sums add 128 exact products in fp32 with
at most 2^-23 of the running sum each, whatever their order; scaling and adding kt of them takes
kt + 2 roundings of 2^-24: (256 + kt + 2) U of the terms' magnitudes, and the type's rounding."""
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def special(cols):
    """Rows of zeros, of one subnormal, of the largest values, of codes and of midpoints of codes."""
    codes = torch.arange(128, dtype=torch.uint8)[:127].view(ref.F8).float()
    mids = (codes[1:] + codes[:-1]) / 2
    fit = lambda v: v.repeat(cols // v.numel() + 1)[:cols]
    rows = [torch.zeros(cols), fit(torch.tensor([1e-44, 0.0])), torch.full((cols,), 3e38), fit(codes), fit(mids),
            -fit(mids), fit(torch.tensor([448.0, 1e-3, -2e-6])), fit(torch.tensor([1.0, float("nan")])),
            fit(torch.tensor([1.0, -float("inf"), 2.0])), torch.full((cols,), 2.0 ** -126)]
    return torch.stack(rows).to(DEV)


@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7168), (3, 127), (5, 128), (6, 136), (7, 257), (33, 1001), (300, 384),
                                       (129, 2048)])
def test_rows(moe, rows, cols, dt):
    for x in (randn(rows, cols).to(dt), randn(rows, cols + 24)[:, 24:].to(dt), randn(rows, cols + 1).to(dt)[:, 1:],
              randn(rows, cols + 8).to(dt)[:, :cols]):
        q, s = moe.moe_quantize_rows_fp8(x)
        wq, ws = ref.quantize_rows(x.float().cpu())
        assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), ws)
        for out in ref.DTYPES:
            v = moe.moe_dequantize_rows_fp8(q, s, cols, out)
            want = (wq.view(ref.F8).float().view(rows, -1, 128) * ws.unsqueeze(-1)).view(rows, -1)[:, :cols].to(out)
            assert torch.equal(v.cpu(), want)


@pytest.mark.parametrize("cols", [128, 200, 1001])
@pytest.mark.parametrize("dt", ref.DTYPES)
def test_special_rows(moe, cols, dt):
    x = special(cols).to(dt)
    q, s = moe.moe_quantize_rows_fp8(x)
    wq, ws = ref.quantize_rows(x.float().cpu())
    assert torch.equal(torch.isnan(s).cpu(), torch.isnan(ws))
    assert torch.equal(torch.nan_to_num(s).cpu(), torch.nan_to_num(ws)) and torch.equal(q.cpu(), wq)
    v = moe.moe_dequantize_rows_fp8(q, s, cols, torch.float32)
    bad = torch.isnan(s).repeat_interleave(128, dim=1)[:, :cols]
    assert torch.equal(torch.isnan(v), bad)


def test_given_outputs_and_perm(moe):
    for cols in (256, 250):
        x = randn(40, cols).bfloat16()
        perm = torch.arange(40, dtype=torch.int32, device=DEV)
        perm[[3, 4, 39]] = -1
        q = torch.full((40, 256), 5, dtype=torch.uint8, device=DEV).view(ref.F8)
        s = torch.full((40, 2), 5.0, device=DEV)
        moe.moe_quantize_rows_fp8(x, q=q, scales=s, perm=perm)
        wq, ws = ref.quantize_rows(x.float().cpu())
        wq[[3, 4, 39]], ws[[3, 4, 39]] = 5, 5.0
        assert torch.equal(q.view(torch.uint8).cpu(), wq) and torch.equal(s.cpu(), ws)


@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (5, 128), (9, 250), (64, 1400), (130, 1001)])
def test_swiglu(moe, rows, cols, dt):
    x = (4 * randn(rows, 2 * cols)).to(dt)
    if rows > 4:  # both ends of silu
        x[0, :cols], x[1, :cols], x[2, :cols], x[3, :cols] = -80.0, 80.0, -1e4, 1e4
    perm = torch.arange(rows, dtype=torch.int32, device=DEV) - (rows > 4) * 1  # row 0 has no pair
    kp = ref.up(cols)
    q = torch.zeros(rows, kp, dtype=torch.uint8, device=DEV)
    s = torch.zeros(rows, kp // 128, device=DEV)
    moe.moe_quantize_rows_fp8(x, q=q, scales=s, swiglu=True, perm=perm)
    a, b = x[:, :cols].double(), x[:, cols:].double()
    y = a * torch.sigmoid(a) * b
    rel = (6 + a.abs().clamp(max=100)) * 2.0 ** -23
    top = torch.nn.functional.pad(y.abs(), (0, kp - cols)).view(rows, -1, 128).amax(dim=-1)
    want = torch.where(top > 0, (top / 448).clamp(min=2.0 ** -126), torch.ones_like(top))
    far = torch.nn.functional.pad(rel * y.abs(), (0, kp - cols)).view(rows, -1, 128).amax(dim=-1) / 448
    live = perm >= 0
    ref.within(s[live], want[live], (far + 2 * ref.U * want + 2.0 ** -126)[live], "scales")
    f = s.double().repeat_interleave(128, dim=1)[:, :cols]
    v = ref.rows64(q, s, cols)
    tol = (2.0 ** -4 + rel + 8 * ref.U) * y.abs() + (2.0 ** -10 + 8 * ref.U) * f + 2.0 ** -126
    ref.within(v[live], y[live], tol[live], "values")
    assert not (~live).any() or (int(q[~live].max()) == 0 and float(s[~live].abs().max()) == 0)
    if rows > 4:
        assert torch.isfinite(v).all()


def test_swiglu_values_that_are_not_finite(moe):
    inf, nan = float("inf"), float("nan")
    a = torch.tensor([[1.0], [-inf], [inf], [nan], [-inf]], device=DEV).expand(5, 128)
    b = torch.tensor([[nan], [2.0], [2.0], [2.0], [inf]], device=DEV).expand(5, 128)
    q, s = moe.moe_quantize_rows_fp8(torch.cat([a, b], 1).contiguous(), swiglu=True)
    assert torch.equal(torch.isnan(s[:, 0]).cpu(), torch.tensor([True, False, True, True, True]))
    assert float(s[1, 0]) == 1.0 and int((q & 127).max()) == 0  # silu(-inf) is -0: a zero code with a sign


@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (1, 128, 128), (2, 130, 250), (3, 256, 384), (2, 1001, 129), (5, 100, 8)])
def test_blocks(moe, E, K, N):
    W = randn(E, K, N).bfloat16()
    W[0, 0, 0] = 300.0
    if E > 2:
        W[1] = 0
        W[2, K // 2, N // 2] = float("inf")
    q, s = moe.moe_quantize_blocks_fp8(W)
    wq, ws = ref.quantize_blocks(W.float().cpu())
    assert torch.equal(torch.nan_to_num(s, nan=-1).cpu(), torch.nan_to_num(ws, nan=-1)) and torch.equal(q.cpu(), wq)
    q2, s2 = moe.moe_quantize_blocks_fp8(W, transpose=False)
    assert torch.equal(torch.nan_to_num(s2, nan=-1), torch.nan_to_num(s.transpose(1, 2), nan=-1))
    assert torch.equal(q2[:, :, :N], q[:, :, :K].transpose(1, 2)) and int(q2[:, :, N:].sum()) == 0


# ------------------------------------------------------------------------------ products
def operands(moe, rows, N, K, E=1, seed=0):
    a = moe.moe_quantize_rows_fp8(randn(rows, K, seed=seed))
    b = moe.moe_quantize_blocks_fp8((randn(E, K, N, seed=seed + 1) * K ** -0.5).bfloat16())
    return a, b


def check_product(got, a, b, K, what):
    """got [rows, N] of 8-bit rows a and one weight matrix b."""
    A, B = ref.rows64(*a, K), ref.weights64(*b, K)
    want, terms = A @ B.t(), A.abs() @ B.abs().t()
    rel, tiny = ref.half_step(got.dtype)
    off = (258 + -(-K // 128)) * ref.U * terms
    ref.within(got, want, off + rel * (want.abs() + off) + tiny, what)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 1), (1, 16, 128), (1, 4096, 7168), (2, 33, 100), (8, 64, 129), (9, 129, 256),
                                      (17, 40, 384), (33, 136, 640), (64, 512, 1000), (65, 1000, 129), (128, 128, 128),
                                      (129, 257, 300), (255, 300, 2000), (300, 2048, 512), (777, 1545, 2700),
                                      (1500, 2500, 384)])
def test_product(moe, rows, N, K, out):
    a, b = operands(moe, rows, N, K)
    o = torch.full((rows, N), 9.0, dtype=out, device=DEV)
    moe.moe_gemm_fp8(*a, *b, o, K)
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    check_product(o, a, (b[0][0], b[1][0]), K, "out")


COUNTS = [[0, 0, 0], [1, 0, 130], [128, 5, 0, 256, 1], [300, 1000, 7, 64, 65, 0, 129], [513, 2, 511, 385]]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(128, 128), (200, 500), (1024, 384)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_product(moe, counts, N, K, out):
    E = len(counts)
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += ref.up(c)
    for rows in (at + 128, max([s + c for s, c in zip(starts, counts) if c] + [1])):
        a, b = operands(moe, rows, N, K, E)
        a[1][:] = torch.where(torch.rand_like(a[1]) < 0.1, torch.zeros_like(a[1]), a[1])
        o = torch.full((rows, N), 9.0, dtype=out, device=DEV)
        moe.moe_gemm_fp8(*a, *b, o, K, counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
        assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
        left = torch.ones(rows, dtype=torch.bool)
        for e, (s, c) in enumerate(zip(starts, counts)):
            if c:
                check_product(o[s:s + c], (a[0][s:s + c], a[1][s:s + c]), (b[0][e], b[1][e]), K, "expert %d" % e)
            left[s:s + c] = False
        assert (o[left.to(DEV)] == 9.0).all()  # rows between the segments


def test_counts_that_do_not_fit(moe):
    a, b = operands(moe, 256, 128, 128, 2)
    o = torch.full((256, 128), 9.0, device=DEV)
    for bad in ([257, 0], [-1, 5], [129, 1], [2 ** 31 - 1, 2 ** 31 - 1]):
        moe.moe_gemm_fp8(*a, *b, o, 128, counts=torch.tensor(bad, dtype=torch.int32, device=DEV))
        assert moe.moe_gemm_fp8_get_error() == moe.MOE_ERR_DEVICE_BOUNDS
        assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
        assert (o == 9.0).all()


def test_values_of_padding_do_not_matter(moe):
    """Codes past K, rows past the last valid one and their scales, NaN among them."""
    K, N = 200, 96
    a, b = operands(moe, 256, N, K, 2)
    counts = torch.tensor([70, 100], dtype=torch.int32, device=DEV)
    o = [torch.zeros(256, N, device=DEV) for _ in range(2)]
    moe.moe_gemm_fp8(*a, *b, o[0], K, counts=counts)
    a[0][:, K:] = 127
    b[0][:, :, K:] = 127
    a[0][70:128], a[1][70:128], a[0][228:], a[1][228:] = 127, float("nan"), 127, float("nan")
    moe.moe_gemm_fp8(*a, *b, o[1], K, counts=counts)
    assert torch.equal(o[0], o[1]) and torch.isfinite(o[1]).all()


def test_nan_stays_in_its_row_and_column(moe):
    a, b = operands(moe, 140, 300, 256)
    a[1][130, 1] = float("nan")
    b[1][0, 1, 0] = float("nan")
    o = torch.zeros(140, 300, device=DEV)
    moe.moe_gemm_fp8(*a, *b, o, 256)
    nan = torch.zeros(140, 300, dtype=torch.bool, device=DEV)
    nan[130], nan[:, 128:256] = True, True
    assert torch.equal(torch.isnan(o), nan)


@pytest.mark.parametrize("N,K", [(500, 1000), (4096, 512)])
def test_rows_do_not_depend_on_the_batch(moe, N, K):
    """One row, a few, a hundred and thousands take different tile shapes: the same bits."""
    a, b = operands(moe, 3000, N, K)
    whole = torch.empty(3000, N, device=DEV)
    moe.moe_gemm_fp8(*a, *b, whole, K)
    for lo, hi in ((0, 1), (5, 21), (100, 228), (512, 1500)):
        o = torch.empty(hi - lo, N, device=DEV)
        moe.moe_gemm_fp8(a[0][lo:hi], a[1][lo:hi], *b, o, K)
        assert torch.equal(o, whole[lo:hi])
    counts = torch.tensor([3000], dtype=torch.int32, device=DEV)
    o = torch.empty(3000, N, device=DEV)
    moe.moe_gemm_fp8(*a, *b, o, K, counts=counts)
    assert torch.equal(o, whole)


def test_unaligned_output_and_stream(moe):
    a, b = operands(moe, 200, 256, 300)
    want = torch.empty(200, 256, device=DEV)
    moe.moe_gemm_fp8(*a, *b, want, 300)
    for dt in (torch.float32, torch.bfloat16):
        for off in (1, 4, 8):
            o = torch.zeros(200 * 256 + 8, dtype=dt, device=DEV)[off:off + 200 * 256].view(200, 256)
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            moe.moe_gemm_fp8(*a, *b, o, 300, stream=side)
            side.synchronize()
            assert torch.equal(o, want.to(dt))


def test_gradient_of_the_rows(moe):
    """dx = dy W^T on the weights in their other order, against the formula and against differences of
    the forward product (linear in x: exact but for rounding)."""
    K, N, rows = 384, 200, 70
    W = (randn(1, K, N) * 0.05).bfloat16()
    fwd, bwd = moe.moe_quantize_blocks_fp8(W), moe.moe_quantize_blocks_fp8(W, transpose=False)
    dy = moe.moe_quantize_rows_fp8(randn(rows, N, seed=4))
    dx = torch.empty(rows, K, device=DEV)
    moe.moe_gemm_fp8(*dy, *bwd, dx, N)
    check_product(dx, dy, (bwd[0][0], bwd[1][0]), N, "dx")
    e = torch.zeros(2, K, device=DEV)
    e[1, 130] = 1.0
    y = torch.empty(2, N, device=DEV)
    moe.moe_gemm_fp8(*moe.moe_quantize_rows_fp8(e), *fwd, y, K)
    num = (y[1] - y[0]).double() @ ref.rows64(*dy, N).t()
    ref.within(dx[:, 130], num, 1e-4, "difference")


def test_graph_replay(moe):
    K, N, E = 512, 384, 4
    a, b = operands(moe, 1024, N, K, E)
    x = randn(1024, K)
    q, s = torch.empty_like(a[0]), torch.empty_like(a[1])
    counts = torch.tensor([10, 300, 0, 129], dtype=torch.int32, device=DEV)
    o = torch.zeros(1024, N, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_quantize_rows_fp8(x, q=q, scales=s)
        moe.moe_gemm_fp8(q, s, *b, o, K, counts=counts)
    for seed, c in ((3, [200, 1, 256, 0]), (4, [10, 300, 0, 129])):
        x.copy_(randn(1024, K, seed=seed))
        counts.copy_(torch.tensor(c, dtype=torch.int32))
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(o)
        moe.moe_gemm_fp8(*moe.moe_quantize_rows_fp8(x), *b, want, K, counts=counts)
        assert torch.equal(o, want) and float(o.abs().max()) > 0
