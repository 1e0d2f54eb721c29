"""Calls around 8-bit experts that the documentation allows at its edges: offsets past 2^31 elements,
every tile shape of the product, two streams at once, workspaces that two captured graphs share,
results in place of operands, and rows that start anywhere.  Tolerances as in the tests of each
operator; what is compared with the same call made otherwise is equal."""
import hashlib
import os
import subprocess
import sys

import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def randn(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


# ------------------------------------------------------------------------- long tensors
def test_rows_past_2_31_values(moe):
    rows, cols = 262200, 8200  # 2.15e9 values, the last block of a row 8 wide
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[:4], x[-4:] = randn(4, cols), randn(4, cols, seed=1)
    x[4:-4] = 0.5
    w = (1 + 0.2 * randn(cols, seed=2)).bfloat16()
    q, s = moe.moe_quantize_rows_fp8(x)
    out, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    moe.moe_rmsnorm(x, w, 1e-6, out=out, rstd=rstd)
    back = moe.moe_dequantize_rows_fp8(q, s, cols)
    for part in (slice(0, 6), slice(rows - 6, rows)):
        wq, wsc = ref.quantize_rows(x[part].float().cpu())
        assert torch.equal(q[part].cpu(), wq) and torch.equal(s[part].cpu(), wsc)
        assert torch.equal(back[part].double().cpu(), ref.rows64(wq, wsc, cols).float().bfloat16().double())
        y, r = ref.norm64(x[part], w, 1e-6)
        ref.within(rstd[part], r, 14 * ref.U * r, "rstd")
        ref.within(out[part], y, (2.0 ** -8 + 16 * ref.U) * 1.01 * y.abs(), "out")
    del back, q, s
    dx, dw = out, torch.empty(cols, device=DEV)  # (the norm is not used again)
    ws = torch.empty(moe.moe_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    moe.moe_rmsnorm_backward(x, x, w, rstd, dx, dw, ws)
    for part in (slice(0, 6), slice(rows - 6, rows)):
        d, _, off, _ = ref.norm_grad64(x[part], x[part], w, rstd[part])
        ref.within(dx[part], d, off + 2.0 ** -8 * (d.abs() + off) + 2.0 ** -134, "dx")


def test_distance_of_rows_past_2_31(moe):
    stride, cols = (1 << 31) + 8, 1000
    x = torch.empty(2 * stride + cols, dtype=torch.bfloat16, device=DEV).as_strided((3, cols), (stride, 1))
    for i in range(3):
        x[i] = randn(cols, seed=i).bfloat16()
    near = x.contiguous()
    got, want = moe.moe_quantize_rows_fp8(x), moe.moe_quantize_rows_fp8(near)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w, a, b = torch.ones(cols, device=DEV), torch.empty_like(near), torch.empty_like(near)
    moe.moe_rmsnorm(x, w, 1e-6, out=a)
    moe.moe_rmsnorm(near, w, 1e-6, out=b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product_past_2_31_outputs(moe, out):
    rows, N, K = 262200, 8200, 128
    a = moe.moe_quantize_rows_fp8(randn(rows, K).bfloat16())
    b = moe.moe_quantize_blocks_fp8(randn(1, K, N, seed=1).bfloat16())
    o = torch.empty(rows, N, dtype=out, device=DEV)
    moe.moe_gemm_fp8(*a, *b, o, K)
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    few = torch.empty(40, N, dtype=out, device=DEV)
    for lo in (0, rows // 2, rows - 40):
        moe.moe_gemm_fp8(a[0][lo:lo + 40], a[1][lo:lo + 40], *b, few, K)
        assert torch.equal(o[lo:lo + 40], few)


def test_weights_past_2_31_values(moe):
    E, K, N = 258, 4096, 2050
    W = torch.empty(E, K, N, dtype=torch.bfloat16, device=DEV).fill_(0.25)
    W[0], W[-1] = randn(K, N), randn(K, N, seed=1)
    for transpose in (True, False):
        q, s = moe.moe_quantize_blocks_fp8(W, transpose=transpose)
        for e in (0, E - 1):
            wq, wsc = ref.quantize_blocks(W[e:e + 1].float().cpu())
            if not transpose:
                wsc = wsc.transpose(1, 2)
                assert torch.equal(q[e, :, :N].t().cpu(), wq[0, :, :K])
            else:
                assert torch.equal(q[e].cpu(), wq[0])
            assert torch.equal(s[e].cpu(), wsc[0])
        if transpose:  # and the last expert's rows through the product
            counts = torch.zeros(E, dtype=torch.int32, device=DEV)
            counts[-1] = 30
            a = moe.moe_quantize_rows_fp8(randn(30, K, seed=3))
            o, want = torch.empty(30, N, device=DEV), torch.empty(30, N, device=DEV)
            moe.moe_gemm_fp8(*a, q, s, o, K, counts=counts)
            moe.moe_gemm_fp8(*a, q[-1].contiguous(), s[-1].contiguous(), want, K)
            assert torch.equal(o, want)


@pytest.mark.parametrize("rows,N,K", [(1, 16384, 7168), (1, 16384, 7040), (5, 16000, 4992), (70, 8192, 7168),
                                      (130, 16384, 2176)])
def test_few_rows_of_long_weights(moe, rows, N, K):
    """Weights from HBM, so that copies land late and out of order; several times, on two sets in turn."""
    a = moe.moe_quantize_rows_fp8(randn(rows, K))
    bs = [moe.moe_quantize_blocks_fp8((randn(1, K, N, seed=i) * K ** -0.5).bfloat16()) for i in (1, 2)]
    outs = [torch.empty(rows, N, device=DEV) for _ in bs]
    for b, o in zip(bs, outs):
        moe.moe_gemm_fp8(*a, *b, o, K)
        A, B = ref.rows64(*a, K), ref.weights64(b[0][0], b[1][0], K)
        ref.within(o, A @ B.t(), (258 + -(-K // 128)) * ref.U * (A.abs() @ B.abs().t()), "out")
    o = torch.empty(rows, N, device=DEV)
    for i in range(20):
        moe.moe_gemm_fp8(*a, *bs[i % 2], o, K)
        assert torch.equal(o, outs[i % 2])
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK


# ------------------------------------------------------------------------- tile shapes
def products(moe):
    """One digest of products of many sizes."""
    h = hashlib.sha256()
    for i, (rows, N, K, E) in enumerate([(1, 33, 128, 1), (9, 500, 1000, 1), (300, 777, 129, 1), (600, 1024, 2100, 1),
                                         (1024, 320, 640, 6), (700, 64, 1300, 3)]):
        a = moe.moe_quantize_rows_fp8(randn(rows, K, seed=i))
        b = moe.moe_quantize_blocks_fp8((randn(E, K, N, seed=i + 50) * K ** -0.5).bfloat16())
        counts = {6: [130, 0, 1, 300, 64, 100], 3: [200, 257, 0]}.get(E)
        counts = torch.tensor(counts, dtype=torch.int32, device=DEV) if counts else None
        for dt in (torch.float32, torch.bfloat16):
            o = torch.zeros(rows, N, dtype=dt, device=DEV)
            moe.moe_gemm_fp8(*a, *b, o, K, counts=counts)
            h.update(o.cpu().view(torch.uint8).numpy().tobytes())
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    return h.hexdigest()


def test_tile_shapes_give_the_same_bits(moe):
    want = products(moe)
    code = "import sys; sys.path[:0] = [%r, %r]\n" % (ROOT, os.path.join(ROOT, "tests")) + \
        "import combine_fp32_router_gb300 as moe, test_gpu_fp8_edges as t; print(t.products(moe))"
    for shape in range(4):
        r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, MOE_FP8_SHAPE=str(shape)),
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        assert r.stdout.split()[-1] == want, "shape %d" % shape


# ------------------------------------------------------------------------- streams and graphs
def test_two_streams_at_once(moe):
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def job(i, T, k, E, d, N):
        x, w = randn(T, d, seed=i).bfloat16(), (1 + 0.1 * randn(d, seed=i + 9))
        idx = torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(i)).to(DEV)
        b = moe.moe_quantize_blocks_fp8((randn(E, d, N, seed=i + 20) * d ** -0.5).bfloat16())
        n = moe.moe_sort_rows_bound(T, k, E)
        i32 = dict(dtype=torch.int32, device=DEV)

        def make():
            return dict(q=torch.zeros(T, d, dtype=torch.uint8, device=DEV), s=torch.zeros(T, d // 128, device=DEV),
                        rows=torch.zeros(n, d, dtype=torch.uint8, device=DEV), rs=torch.zeros(n, d // 128, device=DEV),
                        counts=torch.zeros(E, **i32), perm=torch.zeros(n, **i32), pos=torch.zeros(T, k, **i32),
                        ws=torch.zeros(moe.moe_sort_workspace_bytes(T, E, k), dtype=torch.uint8, device=DEV),
                        y=torch.zeros(n, N, device=DEV), out=torch.zeros(T, N, device=DEV))

        def run(o, stream):
            moe.moe_rmsnorm(x, w, 1e-6, q=o["q"], scales=o["s"], stream=stream)
            moe.moe_sort_tokens(o["q"], idx, o["rows"], o["counts"], o["perm"], o["pos"], o["ws"],
                                x_scales=o["s"], rows_scales=o["rs"], stream=stream)
            moe.moe_gemm_fp8(o["rows"], o["rs"], *b, o["y"], d, counts=o["counts"], stream=stream)
            moe.moe_unsort_tokens(o["y"], None, o["pos"], o["out"], o["ws"], stream=stream)

        return make, run

    jobs = [job(0, 700, 8, 32, 1024, 640), job(1, 90, 4, 16, 2048, 1500)]
    want = []
    for make, run in jobs:
        o = make()
        run(o, None)
        want.append(o)
    got = [[make() for _ in range(4)] for make, _ in jobs]
    torch.cuda.synchronize()
    for turn in range(4):
        for i, (_, run) in enumerate(jobs):
            run(got[i][turn], streams[i])
    torch.cuda.synchronize()
    assert moe.moe_gemm_fp8_get_error() == moe.MOE_OK
    for i in range(2):
        for o in got[i]:
            assert moe.moe_get_error(o["ws"]) == moe.MOE_OK
            for key in ("q", "s", "counts", "perm", "pos", "rows", "y", "out"):
                assert torch.equal(o[key], want[i][key]), key


def test_graphs_that_share_a_workspace(moe):
    rows, cols, T, k, E = 500, 1000, 600, 8, 40
    x = [randn(rows, cols, seed=s).bfloat16() for s in (0, 1)]
    w = torch.ones(cols, device=DEV)
    idx = [torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(s)).to(DEV)
           for s in (0, 1)]
    t = randn(T, 64, seed=3)
    n = moe.moe_sort_rows_bound(T, k, E)
    ws = torch.empty(max(moe.moe_rmsnorm_workspace_bytes(rows, cols), moe.moe_sort_workspace_bytes(T, E, k)),
                     dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)

    def buffers():
        return (torch.zeros(rows, device=DEV), torch.zeros_like(x[0]), torch.zeros_like(x[0]),
                torch.zeros(cols, device=DEV), torch.zeros(n, 64, device=DEV), torch.zeros(E, **i32),
                torch.zeros(n, **i32), torch.zeros(T, k, **i32))

    def run(i, o):
        rstd, out, dx, dw, rows_, counts, perm, pos = o
        moe.moe_rmsnorm(x[i], w, 1e-6, out=out, rstd=rstd)
        moe.moe_rmsnorm_backward(out, x[i], w, rstd, dx, dw, ws)
        moe.moe_sort_tokens(t, idx[i], rows_, counts, perm, pos, ws)

    want, got, graphs = [], [], []
    for i in (0, 1):
        want.append(buffers())
        run(i, want[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        got.append(buffers())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(i, got[i])
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(want[i], got[i]))


# ------------------------------------------------------------------------- in place, anywhere
@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("d", [64, 1001])
def test_row_gradient_in_place(moe, d, dt):
    T, k, E = 130, 4, 8
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(0))
    n = moe.moe_sort_rows_bound(T, k, E)
    pos = ref.sort_ref(idx, E, n)[2].to(DEV)
    rows, dout, gate = randn(n, d).to(dt), randn(T, d, seed=1).to(dt), torch.rand(T, k, device=DEV)
    word = torch.zeros(4, dtype=torch.int32, device=DEV)
    drows, dgate = rows.clone(), torch.empty_like(gate)
    moe.moe_unsort_tokens_backward(dout, rows, gate, pos, drows, dgate, word)
    same, dg2 = rows.clone(), torch.empty_like(gate)
    moe.moe_unsort_tokens_backward(dout, same, gate, pos, same, dg2, word)
    assert torch.equal(same, drows) and torch.equal(dg2, dgate)


@pytest.mark.parametrize("dt", ref.DTYPES + [torch.uint8])
@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("T", [30, 900])
def test_sort_of_rows_that_start_anywhere(moe, T, off, dt):
    k, E, d = 6, 12, 104
    idx = torch.randint(-1, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(T))
    n = moe.moe_sort_rows_bound(T, k, E)
    x = (randn(T * d + off) * 30).abs().to(dt)[off:].view(T, d)
    rows = torch.zeros(n * d + off, dtype=dt, device=DEV)[off:].view(n, d)
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, perm, pos = torch.empty(E, **i32), torch.empty(n, **i32), torch.empty(T, k, **i32)
    ws = torch.empty(moe.moe_sort_workspace_bytes(T, E, k), dtype=torch.uint8, device=DEV)
    moe.moe_sort_tokens(x, idx.to(DEV), rows, counts, perm, pos, ws)
    wc, wp, wpos = ref.sort_ref(idx, E, n)
    assert torch.equal(counts.cpu(), wc) and torch.equal(perm.cpu(), wp) and torch.equal(pos.cpu(), wpos)
    live = wp >= 0
    want = torch.zeros(n, d, dtype=dt)
    want[live] = x.cpu()[wp[live].long() // k]
    assert torch.equal(rows.cpu(), want)
    if dt == torch.uint8:
        return
    out = torch.zeros(T * d + off, dtype=dt, device=DEV)[off:].view(T, d)
    moe.moe_unsort_tokens(rows, None, pos, out, ws)
    pairs = (wpos >= 0).sum(1, keepdim=True).to(DEV)
    full = x.double() * pairs  # k equal terms: every partial sum is a multiple of one value
    ref.within(out, full, ref.half_step(dt)[0] * full.abs() * 1.01 + 2 * k * ref.U * full.abs(), "out")


def test_buffers_are_checked(moe):
    x, pos = torch.zeros(4, 64, device=DEV), torch.full((2, 2), -1, dtype=torch.int32, device=DEV)
    out = torch.empty(2, 64, device=DEV)
    for word in (torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32),
                 torch.zeros(8, dtype=torch.int32, device=DEV)[::2]):
        with pytest.raises(ValueError):
            moe.moe_unsort_tokens(x, None, pos, out, word)
    with pytest.raises(moe.MoeError):  # smaller than moe_rmsnorm_workspace_bytes
        moe.moe_rmsnorm_backward(x, x, x[0], torch.ones(4, device=DEV), x, torch.empty(64, device=DEV),
                                 torch.empty(0, dtype=torch.uint8, device=DEV))
