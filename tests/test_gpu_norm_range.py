"""The norm's gradient of rows that are far from one in size but well inside fp32, their rstd too: the sum
over a row of dy s w leaves fp32's range at both ends there, where n = s rstd is of the order of one and the
gradients are finite and normal.

Tolerances are norm_grad64's: n = s rstd, dy n and <dy n, w> take a rounding each before a row's sum, rstd m
(m = <dy n, w> / cols) two and n once more; dx adds two products to dsum, each rounded once, one of them after
rstd w: no more than 4 |g| + 4 |n m| + 28 |n| mean |g n| in units of rstd 2^-24."""
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_fp32_router_gb300 as m
    return m


def randn(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


# size of s and of dy: sums of dy s w past 3.4e38, dy s below 1e-40, and rstd^2 mean(g n) below 1e-40
@pytest.mark.parametrize("size,grad", [(1e17, 1e20), (1e-16, 1e-25), (1e17, 1e-9)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
# many rows and few, that start on 16 bytes and anywhere, of one warp, of several and of two or four segments a warp
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 1024), (400, 512), (400, 1024), (5, 257), (7, 9000), (300, 9216)])
def test_gradient_of_large_and_small_rows(moe, rows, cols, dt, size, grad):
    s, dy = (randn(rows, cols) * size).to(dt), (randn(rows, cols, seed=1) * grad).to(dt)
    w = (1 + 0.2 * randn(cols, seed=2)).to(dt)
    out, rstd = torch.empty_like(s), torch.empty(rows, device=DEV)
    moe.moe_rmsnorm(s, w, 0.0, out=out, rstd=rstd)
    y, r64 = ref.norm64(s, w, 0.0)
    ref.within(rstd, r64, 14 * ref.U * r64, "rstd")
    ws = torch.empty(moe.moe_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(s), torch.empty(cols, device=DEV)
    moe.moe_rmsnorm_backward(dy, s, w, rstd, dx, dw, ws)
    rx, rw, off, woff = ref.norm_grad64(dy, s, w, rstd)
    rel, tiny = ref.half_step(dt)
    ref.within(dx, rx, off + rel * (rx.abs() + off) + tiny, "dx")
    ref.within(dw, rw, woff + 1e-45, "dw")
