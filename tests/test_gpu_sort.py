"""Tokens sorted by expert and back, and both gradients, on the GPU.

Sorting moves data: equal.  unsort adds k fp32 products in order: k U of the terms' magnitudes, and
the type's rounding.  dgate's sums take 8 steps per segment of 256 of a warp, 5 in the warp and one
per warp.  drows is one fp32 product rounded to the type: equal."""
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def experts(T, k, E, seed=0, drop=0.0, skew=False):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if skew:
        idx[torch.rand(T, k, generator=g) < 0.7] = E // 2
    if drop:
        idx[torch.rand(T, k, generator=g) < drop] = -1
    return idx


def sort(moe, x, idx, E, xs=None, extra=0):
    T, d = x.shape
    k = idx.shape[1]
    n = moe.moe_sort_rows_bound(T, k, E) + extra
    o = dict(rows=torch.full((n, d), 7, device=DEV).to(x.dtype), counts=torch.empty(E, dtype=torch.int32, device=DEV),
             perm=torch.full((n,), 99, dtype=torch.int32, device=DEV), pos=torch.empty(T, k, dtype=torch.int32, device=DEV),
             ws=torch.full((moe.moe_sort_workspace_bytes(T, E, k),), 255, dtype=torch.uint8, device=DEV))
    if xs is not None:
        o["rows_scales"] = torch.full((n, xs.shape[1]), 7.0, device=DEV)
    moe.moe_sort_tokens(x, idx.to(DEV), o["rows"], o["counts"], o["perm"], o["pos"], o["ws"], x_scales=xs,
                        rows_scales=o.get("rows_scales"))
    return o


def check_sort(moe, x, idx, E, o, xs=None):
    assert moe.moe_get_error(o["ws"]) == moe.MOE_OK
    n, k = o["rows"].shape[0], idx.shape[1]
    counts, perm, pos = ref.sort_ref(idx, E, n)
    assert torch.equal(o["counts"].cpu(), counts)
    assert torch.equal(o["perm"].cpu(), perm)
    assert torch.equal(o["pos"].cpu(), pos)
    live = perm >= 0
    for src, dst in ((x, o["rows"]), (xs, o.get("rows_scales"))):
        if src is not None:
            want = torch.full(dst.shape, 7.0).to(dst.dtype)
            want[live] = src.cpu()[perm[live].long() // k]
            assert torch.equal(dst.cpu(), want)


SHAPES = [(0, 2, 4), (1, 1, 1), (1, 8, 256), (3, 2, 5), (64, 8, 16), (255, 8, 1024), (256, 8, 64), (257, 8, 64),
          (1500, 3, 7), (2049, 1, 33), (5000, 16, 1024), (700, 6, 2)]


@pytest.mark.parametrize("T,k,E", SHAPES)
def test_sort(moe, T, k, E):
    for d, dt, drop, skew in ((256, torch.bfloat16, 0.0, False), (33, torch.float16, 0.2, True),
                              (5, torch.uint8, 0.5, False), (129, torch.float32, 1.0, False)):
        x = torch.randint(0, 200, (T, d), device=DEV).to(dt)
        idx = experts(T, k, E, seed=T + d, drop=drop, skew=skew)
        check_sort(moe, x, idx, E, sort(moe, x, idx, E, extra=3 if d == 5 else 0))


@pytest.mark.parametrize("T,k,E,d", [(8, 8, 256, 7168), (300, 8, 64, 1000), (1000, 4, 16, 128)])
def test_sort_8bit_rows(moe, T, k, E, d):
    q, s = moe.moe_quantize_rows_fp8(torch.randn(T, d, device=DEV))
    idx = experts(T, k, E, drop=0.1)
    check_sort(moe, q, idx, E, sort(moe, q, idx, E, xs=s), xs=s)


def test_sort_same_expert_twice_and_one_for_all(moe):
    for T in (40, 900):
        x = torch.randn(T, 64, device=DEV)
        idx = torch.full((T, 4), 3, dtype=torch.int32)
        check_sort(moe, x, idx, 9, sort(moe, x, idx, 9))


@pytest.mark.parametrize("T", [16, 2000])
def test_sort_bad_experts(moe, T):
    x = torch.randn(T, 64, device=DEV)
    idx = experts(T, 2, 8)
    good = idx.clone()
    idx[3, 1], idx[5, 0], idx[T - 1, 1] = 8, -2, 2 ** 31 - 1
    good[3, 1] = good[5, 0] = good[T - 1, 1] = -1
    o = sort(moe, x, idx, 8)
    assert moe.moe_get_error(o["ws"]) == moe.MOE_ERR_DEVICE_BOUNDS
    # the next call clears the record
    moe.moe_sort_tokens(x, good.to(DEV), o["rows"], o["counts"], o["perm"], o["pos"], o["ws"])
    check_sort(moe, x, good, 8, o)


def test_more_than_2_31_bytes(moe):
    T, k, E, d = 40000, 8, 16, 4096  # 2.7 GB of sorted rows
    x = torch.randn(T, d, device=DEV).to(torch.bfloat16)
    idx = experts(T, k, E)
    o = sort(moe, x, idx, E)
    counts, perm, pos = ref.sort_ref(idx, E, o["rows"].shape[0])
    assert torch.equal(o["perm"].cpu(), perm) and torch.equal(o["pos"].cpu(), pos)
    live = (perm >= 0).nonzero().squeeze(1)[::997].to(DEV)
    assert torch.equal(o["rows"][live], x[o["perm"][live].long() // k])
    out, ones = torch.empty_like(x), torch.full((T, k), 1.0 / k, device=DEV)
    moe.moe_unsort_tokens(o["rows"], ones, o["pos"], out, o["ws"])
    assert torch.equal(out, x)  # eight equal terms of an eighth: exact


def unsort64(rows, gate, pos):
    at = pos.clamp(min=0).long()
    y = rows.double()[at] * (pos >= 0).unsqueeze(-1)
    t = y if gate is None else y * gate.double().unsqueeze(-1)
    return y, t.sum(dim=1), t.abs().sum(dim=1)


@pytest.mark.parametrize("dt", ref.DTYPES)
@pytest.mark.parametrize("T,k,E,d", [(1, 1, 1, 8), (1, 8, 64, 7168), (7, 2, 3, 33), (300, 5, 16, 1000),
                                     (129, 16, 64, 264), (1000, 8, 32, 1025), (3, 3, 4, 65536)])
def test_unsort_and_gradients(moe, T, k, E, d, dt):
    idx = experts(T, k, E, drop=0.3)
    n = moe.moe_sort_rows_bound(T, k, E)
    pos = ref.sort_ref(idx, E, n)[2].to(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.randn(n, d, generator=g, device=DEV).to(dt)
    gate = torch.randn(T, k, generator=g, device=DEV)
    dout = torch.randn(T, d, generator=g, device=DEV).to(dt)
    ws = torch.zeros(16, dtype=torch.uint8, device=DEV)
    rel, tiny = ref.half_step(dt)
    out, dx = torch.empty(T, d, dtype=dt, device=DEV), torch.empty(T, d, dtype=dt, device=DEV)
    moe.moe_unsort_tokens(rows, gate, pos, out, ws)
    y, want, terms = unsort64(rows, gate, pos)
    ref.within(out, want, (k + 1) * ref.U * terms + rel * (want.abs() + (k + 1) * ref.U * terms) + tiny, "out")
    moe.moe_sort_tokens_backward(rows, pos, dx, ws)
    _, want, terms = unsort64(rows, None, pos)
    ref.within(dx, want, k * ref.U * terms + rel * (want.abs() + k * ref.U * terms) + tiny, "dx")
    drows, dgate = torch.full_like(rows, 7), torch.empty(T, k, device=DEV)
    moe.moe_unsort_tokens_backward(dout, rows, gate, pos, drows, dgate, ws)
    want_rows = torch.full_like(rows, 7)
    live = pos >= 0
    want_rows[pos[live].long()] = (gate.unsqueeze(-1) * dout.float().unsqueeze(1)).to(dt)[live]
    assert torch.equal(drows, want_rows)
    prod = y * dout.double().unsqueeze(1)
    segs = -(-d // 256)
    steps = 8 * -(-segs // min(segs, 8)) + 5 + 8
    ref.within(dgate, prod.sum(dim=-1), steps * ref.U * prod.abs().sum(dim=-1), "dgate")
    # without the weights' gradient, and in place
    again = torch.full_like(rows, 7)
    moe.moe_unsort_tokens_backward(dout, None, gate, pos, again, None, ws)
    assert torch.equal(again, want_rows)
    again, dg = rows.clone(), torch.empty_like(dgate)
    moe.moe_unsort_tokens_backward(dout, again, gate, pos, again, dg, ws)
    assert torch.equal(again[pos[live].long()], want_rows[pos[live].long()]) and torch.equal(dg, dgate)
    moe.moe_unsort_tokens_backward(dout, None, None, pos, again, None, ws)
    assert torch.equal(again[pos[live].long()], dout.unsqueeze(1).expand(T, k, d)[live])
    assert moe.moe_get_error(ws) == moe.MOE_OK


def test_gate_gradient_against_differences(moe):
    """out is linear in gate and in rows, so differences of the 64-bit form are exact but for rounding."""
    T, k, E, d = 4, 3, 5, 40
    pos = ref.sort_ref(experts(T, k, E, drop=0.2), E, moe.moe_sort_rows_bound(T, k, E))[2].to(DEV)
    rows, gate = torch.randn(moe.moe_sort_rows_bound(T, k, E), d, device=DEV), torch.rand(T, k, device=DEV)
    dout = torch.randn(T, d, device=DEV)
    ws = torch.zeros(16, dtype=torch.uint8, device=DEV)
    drows, dgate = torch.zeros_like(rows), torch.empty(T, k, device=DEV)
    moe.moe_unsort_tokens_backward(dout, rows, gate, pos, drows, dgate, ws)
    f = lambda r, g: float((unsort64(r, g, pos)[1] * dout.double()).sum())
    for t in range(T):
        e = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        e[t, 1] = 0.5
        num = f(rows, gate.double() + e) - f(rows, gate.double() - e)
        assert abs(num - float(dgate[t, 1])) < 1e-4
        if int(pos[t, 1]) >= 0:
            e = torch.zeros(rows.shape, dtype=torch.float64, device=DEV)
            e[int(pos[t, 1]), 3] = 0.5
            num = f(rows.double() + e, gate) - f(rows.double() - e, gate)
            assert abs(num - float(drows[int(pos[t, 1]), 3])) < 1e-5


def test_unsort_bad_rows_and_empty_tokens(moe):
    rows = torch.randn(128, 64, device=DEV)
    pos = torch.tensor([[0, -1], [-1, -1], [128, 5], [-7, 6]], dtype=torch.int32, device=DEV)
    gate = torch.ones(4, 2, device=DEV)
    gate[1] = float("nan")  # the weights of pairs without a row are not used
    out, ws = torch.full((4, 64), 9.0, device=DEV), torch.zeros(16, dtype=torch.uint8, device=DEV)
    moe.moe_unsort_tokens(rows, gate, pos, out, ws)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(out, torch.stack([rows[0], torch.zeros(64, device=DEV), rows[5], rows[6]]))
    ws.zero_()
    drows, dgate = torch.full_like(rows, 7), torch.empty(4, 2, device=DEV)
    moe.moe_unsort_tokens_backward(out, rows, gate, pos, drows, dgate, ws)
    assert moe.moe_get_error(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert (dgate[pos < 0] == 0).all() and float(dgate[2, 0]) == 0
    assert (drows[7:] == 7).all() and (drows[1:5] == 7).all()


@pytest.mark.parametrize("d", [256, 1000, 4096])
def test_tokens_do_not_depend_on_the_batch(moe, d):
    T, k, E = 600, 6, 16
    n = moe.moe_sort_rows_bound(T, k, E)
    pos = ref.sort_ref(experts(T, k, E), E, n)[2].to(DEV)
    rows, gate = torch.randn(n, d, device=DEV).bfloat16(), torch.rand(T, k, device=DEV)
    dout = torch.randn(T, d, device=DEV).bfloat16()
    ws = torch.zeros(16, dtype=torch.uint8, device=DEV)

    def both(lo, hi):
        out, dr, dg = torch.empty_like(dout[lo:hi]), torch.zeros_like(rows), torch.empty(hi - lo, k, device=DEV)
        p, w = pos[lo:hi].contiguous(), gate[lo:hi].contiguous()
        moe.moe_unsort_tokens(rows, w, p, out, ws)
        moe.moe_unsort_tokens_backward(dout[lo:hi].contiguous(), rows, w, p, dr, dg, ws)
        return out, dg

    out, dg = both(0, T)
    for lo, hi in ((0, 1), (17, 90)):
        o, g = both(lo, hi)
        assert torch.equal(o, out[lo:hi]) and torch.equal(g, dg[lo:hi])


def test_streams_and_graphs(moe):
    T, k, E, d = 500, 8, 32, 512
    x = torch.randn(T, d, device=DEV).bfloat16()
    idx = [experts(T, k, E, seed=s) for s in (1, 2)]
    gate = torch.rand(T, k, device=DEV)
    o = sort(moe, x, idx[0], E)
    dev = idx[0].to(DEV)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_sort_tokens(x, dev, o["rows"], o["counts"], o["perm"], o["pos"], o["ws"])
        moe.moe_unsort_tokens(o["rows"], gate, o["pos"], out, o["ws"])
    for i in (0, 1):
        dev.copy_(idx[i])
        o["rows"].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check_sort(moe, x, idx[i], E, o)
        _, want, terms = unsort64(o["rows"], gate, o["pos"])
        ref.within(out, want, 9 * ref.U * terms + 2.0 ** -8 * (want.abs() + 9 * ref.U * terms), "out")
    side = torch.cuda.Stream()
    o["rows"].fill_(7)
    torch.cuda.synchronize()
    moe.moe_sort_tokens(x, dev, o["rows"], o["counts"], o["perm"], o["pos"], o["ws"], stream=side)
    side.synchronize()
    check_sort(moe, x, idx[1], E, o)
