"""Serving one MoE layer with 4-bit experts: the bf16 weights are quantised once to MXFP4; a
prompt's tokens run through the grouped 4-bit products, a few tokens at a time through the
few-token layer, both on the same weights.

    python examples/fp4_experts.py [--tokens T --d D --experts E --topk K --dff F]

Prints the two paths' distance from the bf16 layer and their times.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import combine_fp32_router_gb300 as moe  # noqa: E402
import moe_synth  # noqa: E402


class Fp4Layer:
    """One layer's experts in MXFP4, with its fp32 router [E, d]."""

    def __init__(self, router, W1, W3, W2, k):
        self.router, self.k = router, k
        self.E, self.d, self.dff = W1.shape
        self.W1, self.W3, self.W2 = (moe.moe_quantize_weights_fp4(w) for w in (W1, W3, W2))
        self._ws = {}

    def prompt(self, x):
        """Many tokens: dispatch, quantise the rows, grouped products, combine."""
        T, dev = x.shape[0], x.device
        E, d, k = self.E, self.d, self.k
        logits = x.float() @ self.router.t()
        idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        gate = torch.empty(T, k, device=dev)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm, pos = (torch.empty(T * k, dtype=torch.int32, device=dev) for _ in range(2))
        rows = torch.empty(T * k, d, dtype=torch.bfloat16, device=dev)
        ws = torch.empty(moe.moe_route_workspace_bytes(T, E, k), dtype=torch.uint8, device=dev)
        moe.moe_route_dispatch(x, logits, k, idx, gate, counts, offsets, perm, pos, rows, ws)
        # each expert's rows from a multiple of 128 on (one rank's receive layout)
        plan = moe.moe_ep_plan(counts.cpu().numpy()[None], 0, wave_experts=E)
        first = torch.from_numpy(plan["recv_off"][:, 0].copy()).to(dev)
        n = plan["rows"]
        padded = torch.zeros(n, d, dtype=torch.bfloat16, device=dev)
        err = torch.zeros(4, dtype=torch.int32, device=dev)
        peers = torch.tensor([rows.data_ptr()], dtype=torch.int64, device=dev)
        peer_rows = torch.tensor([T * k], dtype=torch.int64, device=dev)
        rank = torch.zeros(E, dtype=torch.int32, device=dev)
        moe.moe_ep_copy_rows(peers, peer_rows, rank, offsets[:E].contiguous(), first, counts, padded,
                             err)
        xq, xs = moe.moe_quantize_rows_fp4(padded)
        a, b = (torch.zeros(n, self.dff, dtype=torch.float32, device=dev) for _ in range(2))
        moe.moe_gemm_fp4(xq, xs, self.W1[0], self.W1[1], a, d, counts=counts)
        moe.moe_gemm_fp4(xq, xs, self.W3[0], self.W3[1], b, d, counts=counts)
        hq, hs = moe.moe_quantize_rows_fp4(a * torch.sigmoid(a) * b)
        y = torch.zeros(n, d, dtype=torch.bfloat16, device=dev)
        moe.moe_gemm_fp4(hq, hs, self.W2[0], self.W2[1], y, self.dff, counts=counts)
        shift = first - offsets[:E]
        place = (pos.view(T, k) + shift[idx.long()]).to(torch.int32).contiguous()
        out = torch.empty_like(x)
        moe.moe_combine(y, gate, place, out, err)
        for status in (moe.moe_gemm_fp4_get_error(), moe.moe_get_error(err)):
            if status != moe.MOE_OK:
                raise moe.MoeError(status, "Fp4Layer.prompt")
        return out

    def step(self, x):
        """Up to 32 tokens: router, experts and combine in two launches."""
        T = x.shape[0]
        if T not in self._ws:
            self._ws[T] = torch.empty(
                moe.moe_few_workspace_bytes(T, self.d, self.E, self.k, self.dff),
                dtype=torch.uint8, device=x.device)
        out = torch.empty_like(x)
        logits = torch.empty(T, self.E, device=x.device)
        moe.moe_forward_few_fp4(x, logits, self.router, self.W1[0], self.W3[0], self.W2[0],
                                self.W1[1], self.W3[1], self.W2[1], self.k, out, self._ws[T])
        return out


def bf16_layer(x, router, W1, W3, W2, k):
    T, d = x.shape
    E, _, dff = W1.shape
    out = torch.empty_like(x)
    ws = torch.empty(moe.moe_workspace_bytes(T, d, E, k, dff), dtype=torch.uint8, device=x.device)
    moe.moe_forward(x, (x.float() @ router.t()).contiguous(), W1, W3, W2, k, out, ws)
    return out


def distance(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def run(T, d, E, k, dff, few=8, seed=11):
    """Distances from the bf16 layer: of the prompt path, of the few-token path, and of the
    few-token path from the bf16 layer on the weights that the codes stand for."""
    w = moe_synth.custom(T, d, E, k, dff, seed=seed)
    inp = {n: t.to("cuda") for n, t in moe_synth.generate(w).items()}
    g = torch.Generator(device="cuda").manual_seed(seed)
    router = torch.randn(E, d, generator=g, device="cuda") * d ** -0.5
    layer = Fp4Layer(router, inp["W1"], inp["W3"], inp["W2"], k)
    x = inp["x"]
    want = bf16_layer(x, router, inp["W1"], inp["W3"], inp["W2"], k)
    values = [moe.moe_dequantize_rows_fp4(q, s, K).transpose(1, 2).contiguous()
              for (q, s), K in ((layer.W1, d), (layer.W3, d), (layer.W2, dff))]
    few = min(few, T, 32)
    step = layer.step(x[:few].contiguous())
    same = bf16_layer(x[:few].contiguous(), router, *values, k)
    return layer, x, distance(layer.prompt(x), want), distance(step, want[:few]), distance(step, same)


def timed(f, n=20):
    for _ in range(3):
        f()
    e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda.synchronize()
    e[0].record()
    for _ in range(n):
        f()
    e[1].record()
    torch.cuda.synchronize()
    return e[0].elapsed_time(e[1]) * 1000 / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--d", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--dff", type=int, default=1024)
    a = ap.parse_args()
    layer, x, prompt, step, exact = run(a.tokens, a.d, a.experts, a.topk, a.dff)
    print("distance from the bf16 layer: prompt %.3f (4-bit rows and weights), few tokens %.3f "
          "(4-bit weights)" % (prompt, step))
    print("few tokens against the bf16 layer on the quantised weights: %.4f" % exact)
    print("prompt of %d tokens: %.1f us" % (a.tokens, timed(lambda: layer.prompt(x), 5)))
    for T in (1, 8, 32):
        xs = x[:T].contiguous()
        print("%d token(s): %.1f us" % (T, timed(lambda: layer.step(xs))))


if __name__ == "__main__":
    main()
