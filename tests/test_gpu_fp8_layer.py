"""The operators around 8-bit experts as a layer uses them: norm with the residual's addition, router,
tokens sorted by expert, both products with SwiGLU between them, and back; against the same steps in
64 bits on the values that the 8-bit codes stand for."""
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,d,E,k,dff", [(1, 128, 8, 2, 256), (64, 128, 8, 2, 256), (300, 512, 16, 4, 384),
                                         (1000, 256, 5, 3, 128)])
def test_layer(T, d, E, k, dff):
    import combine_fp32_router_gb300 as moe
    g = torch.Generator(device=DEV).manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, res = rnd(T, d).bfloat16(), rnd(T, d).bfloat16()
    w, router = (1 + 0.1 * rnd(d)).bfloat16(), rnd(d, E) * d ** -0.5
    W13, W2 = (rnd(E, d, 2 * dff) * d ** -0.5).bfloat16(), (rnd(E, dff, d) * dff ** -0.5).bfloat16()
    q13, s13 = moe.moe_quantize_blocks_fp8(W13)
    q2, s2 = moe.moe_quantize_blocks_fp8(W2)

    n = moe.moe_sort_rows_bound(T, k, E)
    buf = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=DEV)
    h, q, s = torch.empty_like(x), buf(T, ref.up(d)), buf(T, ref.up(d) // 128, dt=torch.float32)
    moe.moe_rmsnorm(x, w, 1e-6, residual=res, sum_out=res, out=h, q=q, scales=s)
    top, idx = torch.topk(h.float() @ router, k, dim=1)
    gate, idx = torch.softmax(top, dim=1), idx.to(torch.int32)
    rows, rs = buf(n, ref.up(d)), buf(n, ref.up(d) // 128, dt=torch.float32)
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, perm, pos = torch.empty(E, **i32), torch.empty(n, **i32), torch.empty(T, k, **i32)
    ws = buf(moe.moe_sort_workspace_bytes(T, E, k))
    moe.moe_sort_tokens(q, idx, rows, counts, perm, pos, ws, x_scales=s, rows_scales=rs)
    ab = buf(n, 2 * dff, dt=torch.bfloat16)
    moe.moe_gemm_fp8(rows, rs, q13, s13, ab, d, counts=counts)
    hq, hs = buf(n, ref.up(dff)), buf(n, ref.up(dff) // 128, dt=torch.float32)
    moe.moe_quantize_rows_fp8(ab, q=hq, scales=hs, swiglu=True, perm=perm)
    y = buf(n, d, dt=torch.bfloat16)
    moe.moe_gemm_fp8(hq, hs, q2, s2, y, dff, counts=counts)
    out = torch.empty_like(x)
    moe.moe_unsort_tokens(y, gate, pos, out, ws)
    assert moe.moe_get_error(ws) == moe.MOE_OK and moe.moe_gemm_fp8_get_error() == moe.MOE_OK

    # every step in 64 bits from the values that the step before left
    x8, o64, mag = ref.rows64(q, s, d), torch.zeros(T, d, dtype=torch.float64, device=DEV), 0
    mag = torch.zeros_like(o64)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        B13, B2 = ref.weights64(q13[e], s13[e], d), ref.weights64(q2[e], s2[e], dff)
        f = x8[t] @ B13.t()
        r = pos[t, j].long()
        ref.within(ab[r], f, 2.0 ** -8 * f.abs() * 1.01 + 300 * ref.U * (x8[t].abs() @ B13.abs().t()), "first product")
        a, b = ab[r].double().split(dff, dim=1)
        hv = a * torch.sigmoid(a) * b
        h8 = ref.rows64(hq[r], hs[r], dff)
        step = hs[r].double().repeat_interleave(128, dim=1)[:, :dff]
        ref.within(h8, hv, (2.0 ** -4 + 2.0 ** -16) * hv.abs() + 2.0 ** -9.9 * step, "SwiGLU rows")
        yv = h8 @ B2.t()
        ref.within(y[r], yv, 2.0 ** -8 * yv.abs() * 1.01 + 300 * ref.U * (h8.abs() @ B2.abs().t()), "second product")
        o64.index_put_((t,), gate[t, j].double().unsqueeze(1) * y[r].double(), accumulate=True)
        mag.index_put_((t,), (gate[t, j].double().unsqueeze(1) * y[r].double()).abs(), accumulate=True)
    ref.within(out, o64, 2.0 ** -8 * o64.abs() * 1.01 + 2 * (k + 1) * ref.U * mag, "out")
