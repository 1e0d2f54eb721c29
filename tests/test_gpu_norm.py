"""RMS norm with the residual's addition and 8-bit outputs, and its gradient, on the GPU against
64-bit formulas.

Tolerances.  s is one fp32 addition rounded to the type: equal.  The sum of squares passes at most
20 additions of positive terms on its way (8 in a lane, 5 in a warp, 2 + 5 over segments), so rstd is
off by at most (20 + 2) / 2 + 1 roundings and y = s rstd w by two more: 16 U of |y|; the type's own
rounding is added.  The 8-bit form is a function of the fp32 y, which is `out` in fp32: equal."""
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def make(rows, cols, dt, seed=0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g, device=DEV).to(dt)[:, pad:]
    r = torch.randn(rows, cols, generator=g, device=DEV).to(dt)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(dt)
    return x, r, w


def run(moe, x, w, r=None, eps=EPS, fp8=True, out=True, **kw):
    rows, cols = x.shape
    o = dict(out=torch.empty(rows, cols, dtype=x.dtype, device=DEV) if out else None,
             q=torch.full((rows, ref.up(cols)), 77, dtype=torch.uint8, device=DEV) if fp8 else None,
             scales=torch.empty(rows, ref.up(cols) // 128, device=DEV) if fp8 else None,
             sum_out=torch.empty(rows, cols, dtype=x.dtype, device=DEV) if r is not None else None,
             rstd=torch.empty(rows, device=DEV))
    o.update(kw)
    moe.moe_rmsnorm(x, w, eps, residual=r, **o)
    return o


def check(x, w, r, o, eps=EPS):
    dt = x.dtype
    s = x if r is None else (x.float() + r.float()).to(dt)
    if r is not None:
        assert torch.equal(o["sum_out"], s)
    y, rstd = ref.norm64(s, w, eps)
    rel, tiny = ref.half_step(dt)
    ref.within(o["rstd"], rstd, 14 * ref.U * rstd, "rstd")
    if o["out"] is not None:
        ref.within(o["out"], y, (rel + 16 * ref.U) * y.abs() * (1 + rel) + tiny, "out")
    if o["q"] is not None:
        cols = x.shape[1]
        if dt == torch.float32 and o["out"] is not None:
            q, sc = ref.quantize_rows(o["out"].cpu())
            assert torch.equal(o["q"].cpu(), q)
            assert torch.equal(o["scales"].cpu(), sc)
        else:
            # a code is off by half a step of E4M3: 2^-4 of the value, or 2^-10 below the normals
            v = ref.rows64(o["q"], o["scales"], cols)
            f = o["scales"].double().repeat_interleave(128, dim=1)[:, :cols]
            ref.within(v, y, (2.0 ** -4 + 32 * ref.U) * y.abs() + (2.0 ** -10 + 32 * ref.U) * f, "q")
            top = ref.quantize_rows(y.float().cpu())[1]
            ref.within(o["scales"], top, 20 * ref.U * top.abs(), "scales")
        assert int(o["q"][:, cols:].max() if cols % 128 else 0) == 0  # zero codes past the row


@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("cols", [1, 7, 8, 128, 136, 255, 256, 257, 1000, 1925, 2048, 7168, 8200, 16384])
@pytest.mark.parametrize("rows", [1, 5, 160])
def test_forward(moe, rows, cols, dt):
    x, r, w = make(rows, cols, dt, seed=rows + cols)
    check(x, w, r, run(moe, x, w, r))
    check(x, w, None, run(moe, x, w))
    check(x, w.float(), None, run(moe, x, w.float(), out=dt == torch.float32))


@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("pad", [1, 8, 24])
def test_strided_and_unaligned_rows(moe, dt, pad):
    x, r, w = make(33, 512, dt, pad=pad)
    check(x, w, r, run(moe, x, w, r))


def test_no_rows(moe):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    run(moe, x, torch.ones(256, dtype=torch.bfloat16, device=DEV))
    dw = torch.ones(256, device=DEV)
    ws = torch.empty(moe.moe_rmsnorm_workspace_bytes(0, 256), dtype=torch.uint8, device=DEV)
    moe.moe_rmsnorm_backward(x, x, dw, torch.empty(0, device=DEV), torch.empty_like(x), dw.fill_(3), ws)
    assert float(dw.abs().max()) == 0


def test_in_place_residual(moe):
    x, r, w = make(300, 2048, torch.bfloat16)
    want = run(moe, x, w, r)
    s = r.clone()
    got = run(moe, x, w, s, sum_out=s)
    assert torch.equal(s, want["sum_out"]) and torch.equal(got["q"], want["q"])
    s = x.clone()
    got = run(moe, s, w, r, sum_out=s)
    assert torch.equal(s, want["sum_out"]) and torch.equal(got["out"], want["out"])


@pytest.mark.parametrize("cols", [200, 1000, 7168])
def test_rows_do_not_depend_on_the_batch(moe, cols):
    x, r, w = make(700, cols, torch.bfloat16)
    whole = run(moe, x, w, r)
    for lo, hi in ((0, 1), (3, 5), (100, 500)):
        part = run(moe, x[lo:hi].contiguous(), w, r[lo:hi].contiguous())
        for k in ("out", "q", "scales", "sum_out", "rstd"):
            assert torch.equal(part[k], whole[k][lo:hi]), k


def test_odd_values(moe):
    x, _, w = make(6, 384, torch.float32)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    x[3] = x[3] * 1e-30  # rstd is 1 / sqrt(eps)
    x[4] = 0
    x[4, 7] = 1e-38
    o = run(moe, x, w)
    check(x[[0, 3, 5]], w, None, {k: (v[[0, 3, 5]] if v is not None else None) for k, v in o.items()})
    assert torch.isnan(o["out"][1]).all() and torch.isnan(o["scales"][1]).all()
    assert torch.isnan(o["out"][2, 300]) and torch.isnan(o["scales"][2, 2])
    assert int(o["q"][2, 256:].max()) == 0  # a block without a scale has zero codes
    assert torch.equal(o["scales"][0], torch.ones(3, device=DEV))
    q, s = ref.quantize_rows(o["out"][4:5].cpu())
    assert torch.equal(o["q"][4:5].cpu(), q) and torch.equal(o["scales"][4:5].cpu(), s)
    z = run(moe, x[:1], w, eps=0.0)  # 0 / 0
    assert torch.isnan(z["out"]).all()


def grads(moe, dy, s, w, rstd, dsum=None, dx=None):
    rows, cols = dy.shape
    ws = torch.full((moe.moe_rmsnorm_workspace_bytes(rows, cols),), 255, dtype=torch.uint8, device=DEV)
    dx = torch.empty_like(dy) if dx is None else dx
    dw = torch.empty(cols, device=DEV)
    moe.moe_rmsnorm_backward(dy, s, w, rstd, dx, dw, ws, dsum=dsum)
    return dx, dw


@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("cols", [1, 9, 128, 256, 777, 1024, 1925, 4096, 8200, 16384])
@pytest.mark.parametrize("rows", [1, 7, 200, 1300])
def test_backward(moe, rows, cols, dt):
    s, dsum, w = make(rows, cols, dt, seed=rows * 3 + cols)
    dy = make(rows, cols, dt, seed=5)[0]
    rstd = run(moe, s, w, fp8=False)["rstd"]
    rel, tiny = ref.half_step(dt)
    for ds, ww in ((None, w), (dsum, w.float())):
        dx, dw = grads(moe, dy, s, ww, rstd, ds)
        rx, rw, off, woff = ref.norm_grad64(dy, s, ww, rstd, ds)
        ref.within(dx, rx, off + rel * (rx.abs() + off) + tiny, "dx")
        ref.within(dw, rw, woff + 1e-45, "dw")


def test_backward_in_place_and_without_weights(moe):
    s, dsum, w = make(500, 1536, torch.bfloat16)
    dy = make(500, 1536, torch.bfloat16, seed=5)[0]
    rstd = run(moe, s, w, fp8=False)["rstd"]
    dx, dw = grads(moe, dy, s, w, rstd, dsum)
    for i in range(3):
        a = [dy.clone(), s.clone(), dsum.clone()]
        got, dw2 = grads(moe, a[0], a[1], w, rstd, a[2], dx=a[i])
        assert torch.equal(got, dx) and torch.equal(dw2, dw)
    only = torch.empty_like(dy)
    moe.moe_rmsnorm_backward(dy, s, w, rstd, only, None, None, dsum=dsum)
    assert torch.equal(only, dx)


def test_backward_against_differences(moe):
    """The formula's gradient of sum(dy y) by central differences in 64 bits: their error is of the
    order of h^2 times the third derivative (below 1e-8 here), the kernel's of fp32."""
    s, _, w = make(3, 40, torch.float32, seed=9)
    dy = make(3, 40, torch.float32, seed=10)[0]
    rstd = run(moe, s, w, fp8=False)["rstd"]
    dx, dw = grads(moe, dy, s, w, rstd)
    f = lambda a, b: float((ref.norm64(a, b, EPS)[0] * dy.double()).sum())
    h = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 39)):
        d = torch.zeros(3, 40, dtype=torch.float64, device=DEV)
        d[i, j] = h
        num = (f(s.double() + d, w) - f(s.double() - d, w)) / (2 * h)
        assert abs(num - float(dx[i, j])) < 1e-5 * (1 + abs(num))
        e = d[i]
        num = (f(s, w.double() + e) - f(s, w.double() - e)) / (2 * h)
        assert abs(num - float(dw[j])) < 1e-5 * (1 + abs(num))


def test_streams_and_graphs(moe):
    x, r, w = make(64, 7168, torch.bfloat16)
    dy = make(64, 7168, torch.bfloat16, seed=5)[0]
    want = run(moe, x, w, r)
    wdx, wdw = grads(moe, dy, want["sum_out"], w, want["rstd"])
    side = torch.cuda.Stream()
    o = {k: torch.zeros_like(v) for k, v in want.items()}
    ws = torch.empty(moe.moe_rmsnorm_workspace_bytes(64, 7168), dtype=torch.uint8, device=DEV)
    dx, dw = torch.zeros_like(dy), torch.zeros(7168, device=DEV)
    torch.cuda.synchronize()
    moe.moe_rmsnorm(x, w, EPS, residual=r, stream=side, **o)
    side.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in o)
    x2 = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_rmsnorm(x2, w, EPS, residual=r, **o)
        moe.moe_rmsnorm_backward(dy, o["sum_out"], w, o["rstd"], dx, dw, ws)
    for seed in (1, 0):
        x2.copy_(make(64, 7168, torch.bfloat16, seed=seed)[0])
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in o)
    assert torch.equal(dx, wdx) and torch.equal(dw, wdw)
