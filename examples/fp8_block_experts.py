"""One pre-norm MoE layer with 8-bit experts (a scale per 128 values), forward and the gradients of
its inputs: norm with the residual's addition, router, tokens sorted by expert, both products with
SwiGLU between them, and back.

    python examples/fp8_block_experts.py [--tokens T --d D --experts E --topk K --dff F]

Prints how far 8 bits take the output and the gradients from the same layer in fp32 on the weights
that the codes stand for, and the times.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import combine_fp32_router_gb300 as moe  # noqa: E402

EPS = 1e-6


def new(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Fp8Layer:
    """W13 [E, d, 2 dff] (gate and up side by side) and W2 [E, dff, d] bf16, quantised once in both
    orders: over their rows for the products, over their columns for the gradients."""

    def __init__(self, weight, router, W13, W2, k):
        self.weight, self.router, self.k = weight, router, k  # [d], [E, d]
        self.E, self.dff, self.d = W2.shape
        self.W13, self.W2 = (moe.moe_quantize_blocks_fp8(w) for w in (W13, W2))
        self.W13t, self.W2t = (moe.moe_quantize_blocks_fp8(w, transpose=False) for w in (W13, W2))

    def forward(self, x, residual):
        """(out, s): s = x + residual is what the next layer adds to."""
        T, d, dff, E, k = x.shape[0], self.d, self.dff, self.E, self.k
        kd, kf = moe.moe_fp8_row_bytes(d), moe.moe_fp8_row_bytes(dff)
        u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
        s, h, rstd = torch.empty_like(x), torch.empty_like(x), new(T)
        q, qs = new(T, kd, dtype=u8), new(T, kd // 128)
        moe.moe_rmsnorm(x, self.weight, EPS, residual=residual, sum_out=s, out=h, q=q, scales=qs, rstd=rstd)
        top, idx = torch.topk(h.float() @ self.router.t(), k, dim=1)
        gate, idx = torch.softmax(top, dim=1), idx.to(i32)
        n = moe.moe_sort_rows_bound(T, k, E)
        rows, rs = new(n, kd, dtype=u8), new(n, kd // 128)
        counts, perm, pos = new(E, dtype=i32), new(n, dtype=i32), new(T, k, dtype=i32)
        ws = new(moe.moe_sort_workspace_bytes(T, E, k), dtype=u8)
        moe.moe_sort_tokens(q, idx, rows, counts, perm, pos, ws, x_scales=qs, rows_scales=rs)
        ab = new(n, 2 * dff, dtype=bf)
        moe.moe_gemm_fp8(rows, rs, *self.W13, ab, d, counts=counts)
        hq, hs = new(n, kf, dtype=u8), new(n, kf // 128)
        moe.moe_quantize_rows_fp8(ab, q=hq, scales=hs, swiglu=True, perm=perm)
        y, out = new(n, d, dtype=bf), torch.empty_like(x)
        moe.moe_gemm_fp8(hq, hs, *self.W2, y, dff, counts=counts)
        moe.moe_unsort_tokens(y, gate, pos, out, ws)
        self.kept = (s, h, rstd, gate, idx, counts, perm, pos, ws, ab, y)
        return out, s

    def backward(self, dout, ds):
        """Gradient of x (and of residual) and of the norm's weight, for gradients of out and s."""
        s, h, rstd, gate, idx, counts, perm, pos, ws, ab, y = self.kept
        T, d, dff, n = s.shape[0], self.d, self.dff, y.shape[0]
        dy, dgate = torch.empty_like(y), torch.empty_like(gate)
        moe.moe_unsort_tokens_backward(dout, y, gate, pos, dy, dgate, ws)
        dyq, dys = self._rows(dy, perm)
        dh = new(n, dff)
        moe.moe_gemm_fp8(dyq, dys, *self.W2t, dh, d, counts=counts)
        a, b = ab.float().split(dff, dim=1)
        sig = torch.sigmoid(a)
        dab = torch.cat([dh * b * sig * (1 + a * (1 - sig)), dh * a * sig], dim=1).bfloat16()
        dabq, dabs = self._rows(dab, perm)
        drows, dnorm = new(n, d, dtype=torch.bfloat16), torch.empty_like(s)
        moe.moe_gemm_fp8(dabq, dabs, *self.W13t, drows, 2 * dff, counts=counts)
        moe.moe_sort_tokens_backward(drows, pos, dnorm, ws)
        # the router: softmax over the chosen, then the logits' rows
        dtop = gate * (dgate - (gate * dgate).sum(dim=1, keepdim=True))
        dlogits = torch.zeros(T, self.E, device="cuda").scatter_(1, idx.long(), dtop)
        dnorm = (dnorm.float() + dlogits @ self.router).bfloat16()
        dx, dweight = torch.empty_like(s), new(d)
        moe.moe_rmsnorm_backward(dnorm, s, self.weight, rstd, dx, dweight,
                                 new(moe.moe_rmsnorm_workspace_bytes(T, d), dtype=torch.uint8), dsum=ds)
        for status in (moe.moe_gemm_fp8_get_error(), moe.moe_get_error(ws)):
            if status != moe.MOE_OK:
                raise moe.MoeError(status, "Fp8Layer.backward")
        return dx, dweight

    @staticmethod
    def _rows(t, perm):
        """8-bit rows of sorted rows; those without a pair are left out."""
        k = moe.moe_fp8_row_bytes(t.shape[1])
        q, s = new(t.shape[0], k, dtype=torch.uint8), new(t.shape[0], k // 128)
        return moe.moe_quantize_rows_fp8(t, q=q, scales=s, perm=perm)


def plain(x, residual, weight, router, W13, W2, idx):
    """The layer in fp32 with the experts `idx` [T, k]: (out, s)."""
    s = x + residual
    h = s * torch.rsqrt(s.square().mean(dim=1, keepdim=True) + EPS) * weight
    gate = torch.softmax((h @ router.t()).gather(1, idx.long()), dim=1)
    out = torch.zeros_like(x)
    for e in range(W2.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        a, b = (h[t] @ W13[e]).chunk(2, dim=1)
        y = (torch.nn.functional.silu(a) * b) @ W2[e]
        out = out.index_add(0, t, gate[t, j].unsqueeze(1) * y)
    return out, s


def distance(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def build(T, d, E, k, dff, seed=11):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    layer = Fp8Layer((1 + 0.1 * rnd(d)).bfloat16(), rnd(E, d) * d ** -0.5,
                     (rnd(E, d, 2 * dff) * d ** -0.5).bfloat16(), (rnd(E, dff, d) * dff ** -0.5).bfloat16(), k)
    return layer, [rnd(T, d).bfloat16() for _ in range(4)]


def run(T, d, E, k, dff):
    """Distances from the plain layer: of the output, of x's gradient and of the weight's."""
    layer, (x, residual, dout, ds) = build(T, d, E, k, dff)
    out, _ = layer.forward(x, residual)
    dx, dweight = layer.backward(dout, ds)
    W13, W2 = (torch.stack([moe.moe_dequantize_rows_fp8(q[e], s[e].repeat_interleave(128, dim=0)[:q.shape[1]].contiguous(),
                                                        K, dtype=torch.float32).t() for e in range(E)])
               for (q, s), K in ((layer.W13, d), (layer.W2, dff)))
    leaf, w = x.float().requires_grad_(), layer.weight.float().requires_grad_()
    want, s = plain(leaf, residual.float(), w, layer.router, W13, W2, layer.kept[4])
    torch.autograd.backward([want, s], [dout.float(), ds.float()])
    return distance(out, want.detach()), distance(dx, leaf.grad), distance(dweight, w.grad)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--d", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--dff", type=int, default=1024)
    a = ap.parse_args()
    sizes = a.tokens, a.d, a.experts, a.topk, a.dff
    print("distance from the layer in fp32: output %.3f, gradient of x %.3f, of the norm's weight %.3f" % run(*sizes))
    layer, (x, residual, dout, ds) = build(*sizes)
    for name, f in (("forward", lambda: layer.forward(x, residual)), ("backward", lambda: layer.backward(dout, ds))):
        for _ in range(3):
            f()
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        torch.cuda.synchronize()
        e[0].record()
        for _ in range(20):
            f()
        e[1].record()
        torch.cuda.synchronize()
        print("%s: %.0f us" % (name, e[0].elapsed_time(e[1]) * 50))


if __name__ == "__main__":
    main()
