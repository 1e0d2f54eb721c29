"""Workloads of the 4-bit expert operators: microscaled quantisation, the product of two
quantised matrices, and the whole layer for a few tokens on quantised experts.

Every workload runs in two ways.  With ``own`` false, ``run`` computes the operator from
elementary torch operations in 32 bits; with ``own`` true it makes the calls a user of the
library makes.  ``exact`` computes the same outputs in 64 bits, written separately.

Format (OCP Microscaling Formats 1.0, MXFP4): blocks of 32 consecutive values along a row
share a scale 2^(s - 127), s = floor(log2(amax)) - 2 + 127 held in [0, 254]; each value is
an E2M1 number (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to x / scale, ties to
the even mantissa, saturating at 6.  A row of C values takes round_up(C, 128) / 2 bytes (low
nibble first); the scale bytes of 128 rows x 4 blocks lie together in 512 bytes, row r and
block b at (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4, the tiles ordered by (r // 128, b // 4).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def listed():
    return [
        # -- quantisation of rows and back: the activations of a layer before its products
        # one decode step's tokens at the large layer's width: latency
        dict(name="rows_decode", op="rows", rows=8, cols=7168, dtype="bf16"),
        # ragged: an odd token count, a width that ends inside a block, fp32 activations that
        # are a column slice of a wider matrix
        dict(name="rows_ragged_f32", op="rows", rows=1003, cols=1925, dtype="f32", pad=11),
        # a prefill batch at the large layer's width: bandwidth
        dict(name="rows_prefill", op="rows", rows=16384, cols=7168, dtype="bf16", pad=0),
        # -- expert weights [E, K, N], quantised along K into [E, N, K]: loading a checkpoint
        dict(name="weights_mid", op="weights", E=32, K=2048, N=1024),
        # -- products of quantised rows and quantised weights
        # three tokens through a projection of the large layer: weight streaming
        dict(name="gemm_three_rows", op="gemm", rows=3, N=4096, K=7168, E=1, out="bf16"),
        # ragged in every size
        dict(name="gemm_ragged", op="gemm", rows=777, N=1545, K=2976, E=1, out="bf16"),
        # the first projection of the mid layer's experts, 24576 token-expert pairs over 64
        # experts with unequal shares (some empty)
        dict(name="gemm_experts_mid", op="gemm", rows=24576, N=1024, K=2048, E=64, out="bf16"),
        # a dense projection of a prefill batch: tensor-core rate
        dict(name="gemm_prefill", op="gemm", rows=8192, N=7168, K=7168, E=1, out="bf16"),
        # -- the whole layer for a few tokens: router, experts, combine
        # a small layer: launch and synchronisation latency alone
        dict(name="few_tiny", op="few", T=8, d=128, E=8, k=2, dff=256, router=True),
        # single-token decode of the large layer
        dict(name="few_one_token", op="few", T=1, d=7168, E=256, k=8, dff=2048, router=True),
        # the largest batch of the mid layer, with the router's logits already there
        dict(name="few_mid_32", op="few", T=32, d=2048, E=64, k=6, dff=1024, router=False),
        # a small serving batch of the large layer
        dict(name="few_large_16", op="few", T=16, d=7168, E=256, k=8, dff=2048, router=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "weights", "gemm", "gemm", "few", "few"])
    if op == "rows":
        cols = _log_int(rng, 33, 8192)
        rows = _log_int(rng, 1, min(65536, 16384 * 7168 // cols))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, pad=rng.choice([0, 0, 1, 24]))
    if op == "weights":
        K = 128 * rng.choice([1, 2, 3, 5, 8, 11, 16, 20, 28, 32, 40])
        N = 128 * rng.randint(1, 20)
        return dict(op=op, E=rng.randint(1, max(1, min(64, (64 << 20) // (K * N)))), K=K, N=N)
    if op == "gemm":
        N, K = _log_int(rng, 64, 7168), _log_int(rng, 64, 7168)
        if rng.random() < 0.4:
            E = rng.randint(2, 64)
            rows = _log_int(rng, 1, 24576)
            while 2.0 * rows * N * K > 2.0 * 8192 * 7168 * 7168 or E * N * K > 64 * 2048 * 1024:
                rows, N, K = max(1, rows // 2), max(64, N * 2 // 3), max(64, K * 2 // 3)
        else:
            E = 1
            rows = _log_int(rng, 1, 8192)
        return dict(op=op, rows=rows, N=N, K=K, E=E, out=rng.choice(["bf16", "bf16", "f32"]))
    d = 128 * rng.choice([1, 2, 3, 5, 7, 9, 13, 16, 21, 28, 32, 40, 56])
    dff = 128 * _log_int(rng, 1, 16)
    E = _log_int(rng, 1, 256)
    k = rng.randint(1, min(E, 8))
    T = _log_int(rng, 1, 32)
    while T * k * d * dff > 16 * 8 * 7168 * 2048:
        T = max(1, T // 2)
    return dict(op=op, T=T, d=d, E=E, k=k, dff=dff, router=rng.random() < 0.7)


def _up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------------- the plain format
def _plain_scale_exp(x):
    """Shared exponents [R, B] (the unbiased s - 127) of x [R, B, 32] fp32."""
    amax = x.abs().amax(dim=-1)
    _, e = torch.frexp(amax)  # amax = m 2^e, m in [.5, 1)
    e = torch.where(amax > 0, e - 3, torch.full_like(e, -127))
    return e.clamp(-127, 125)


def _plain_round(v):
    """The nearest E2M1 value of v, ties to even, saturating."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _blocks(x, cols):
    """x [..., C] as fp32 blocks [..., round_up(C, 128) / 32, 32], zeros at the end."""
    kp = _up(cols, 128)
    x = x.float()
    if kp != cols:
        x = torch.nn.functional.pad(x, (0, kp - cols))
    return x.reshape(*x.shape[:-1], kp // 32, 32)


def _plain_quantize(x):
    """Values [..., C] fp32 that x [..., C] stands for after quantisation along its last
    dimension."""
    C = x.shape[-1]
    b = _blocks(x, C)
    e = _plain_scale_exp(b).unsqueeze(-1)
    q = torch.ldexp(_plain_round(torch.ldexp(b, -e)), e)
    return q.reshape(*x.shape[:-1], _up(C, 128))[..., :C]


def _encode(x):
    """Packed codes [R, Kp / 2] and tiled scale bytes of x [R, C] fp32."""
    R, C = x.shape
    b = _blocks(x, C)
    e = _plain_scale_exp(b)
    q = _plain_round(torch.ldexp(b, -e.unsqueeze(-1)))
    a = q.abs()
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, a + 1)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    code = code.reshape(R, -1, 2)
    packed = code[..., 0] | (code[..., 1] << 4)
    rp = _up(R, 128)
    s = torch.zeros(rp, e.shape[1], dtype=torch.uint8, device=x.device)
    s[:R] = (e + 127).to(torch.uint8)
    s = s.reshape(rp // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return packed.contiguous(), s


def _decode_values(packed):
    """E2M1 values [..., K] fp32 of packed codes [..., K / 2]."""
    code = torch.stack([packed & 15, packed >> 4], dim=-1).reshape(*packed.shape[:-1], -1)
    m = (code & 7).float()
    v = torch.where(m <= 4, 0.5 * m, torch.where(m < 7, m - 2, m - 1))
    return torch.where(code >= 8, -v, v)


def _decode_scales(s, rows, kp):
    """Scale factors [..., rows, kp / 32] fp32 of tiled scale bytes [..., bytes]."""
    lead = s.shape[:-1]
    # (row tile, k tile, r % 32, r // 32, block) -> (row tile, r // 32, r % 32, k tile, block)
    s = s.reshape(*lead, -1, kp // 128, 32, 4, 4).transpose(-4, -2)
    s = s.reshape(*lead, -1, kp // 32)[..., :rows, :]
    return torch.exp2(s.float() - 127.0)


def _dequantize(packed, s, rows, K):
    """fp32 values [..., rows, K]."""
    kp = packed.shape[-1] * 2
    v = _decode_values(packed).reshape(*packed.shape[:-1], kp // 32, 32)
    v = v * _decode_scales(s, rows, kp).unsqueeze(-1)
    return v.reshape(*packed.shape[:-1], kp)[..., :K]


# ------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _activations(g, rows, cols):
    """Normal values with a few channels several times larger, as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    boost = torch.rand(cols, generator=g, device=DEV) < 0.01
    return x * torch.where(boost, 12.0, 1.0)


def _quantized_weights(g, E, N, K):
    """Weights [E, N, K] ~ N(0, 1/sqrt(K)) as packed codes [E, N, Kp / 2] and scale bytes
    [E, bytes]."""
    kp, per = _up(K, 128), max(1, (1 << 28) // (_up(N, 128) * _up(K, 128)))
    q = torch.empty(E, N, kp // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(E, _up(N, 128) * kp // 32, dtype=torch.uint8, device=DEV)
    np_ = _up(N, 128)
    for e in range(0, E, per):
        n = min(per, E - e)
        w = torch.zeros(n, np_, K, device=DEV)
        w[:, :N] = torch.randn(n, N, K, generator=g, device=DEV) * K ** -0.5
        a, b = _encode(w.reshape(n * np_, K))
        q[e:e + n] = a.reshape(n, np_, -1)[:, :N]
        s[e:e + n] = b.reshape(n, -1)
    return q, s


def _shares(case, seed):
    """Rows of each expert: unequal, some zero, adding up to case["rows"]."""
    E, rows = case["E"], case["rows"]
    if E == 1:
        return [rows]
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(E, generator=g) ** 2 * (torch.rand(E, generator=g) > 0.05)
    if float(w.sum()) == 0:
        w[0] = 1.0
    c = torch.floor(w / w.sum() * rows).to(torch.int64)
    c[int(torch.argmax(w))] += rows - int(c.sum())
    return c.tolist()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "rows":
        pad = case.get("pad", 0)
        x = _activations(g, case["rows"], case["cols"] + pad).to(DTYPES[case["dtype"]])
        st["x"] = x[:, :case["cols"]]  # pad > 0: rows with a stride, not contiguous
    elif op == "weights":
        E, K, N = case["E"], case["K"], case["N"]
        st["W"] = (torch.randn(E, K, N, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
    elif op == "gemm":
        E, N, K = case["E"], case["N"], case["K"]
        counts = _shares(case, seed)
        # a buffer that holds the experts' segments, each from a multiple of 128 rows on,
        # however the rows fall
        rows = case["rows"] if E == 1 else _up(case["rows"], 128) + 128 * E
        st["aq"], st["a_scales"] = _encode(_activations(g, rows, K))
        st["bq"], st["b_scales"] = _quantized_weights(g, E, N, K)
        st["rows"] = rows
        if E > 1:
            st["counts"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
            first, at = [], 0
            for c in counts:
                first.append(at)
                at += _up(c, 128)
            cap = max(counts)
            # for each expert, the rows of its segment (the first row again past its end) and
            # which of them it has
            n = torch.arange(cap, device=DEV)
            cnt = st["counts"].long()
            st["has"] = n[None, :] < cnt[:, None]
            st["seg"] = torch.tensor(first, device=DEV)[:, None] + n[None, :] * st["has"]
            st["seg"] = st["seg"].clamp(max=rows - 1)
            st["live"] = st["seg"][st["has"]]
        st["out"] = torch.zeros(rows, N, dtype=DTYPES[case["out"]], device=DEV)
    else:
        T, d, E, dff = case["T"], case["d"], case["E"], case["dff"]
        st["x"] = _activations(g, T, d).to(torch.bfloat16)
        st["router"] = torch.randn(E, d, generator=g, device=DEV) * d ** -0.5
        st["logits"] = torch.randn(T, E, generator=g, device=DEV)
        st["W1"] = _quantized_weights(g, E, dff, d)
        st["W3"] = _quantized_weights(g, E, dff, d)
        st["W2"] = _quantized_weights(g, E, d, dff)
        st["out"] = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------------------- one pass
def _plain_gemm(st, case):
    N, K, E = case["N"], case["K"], case["E"]
    a = _dequantize(st["aq"], st["a_scales"], st["rows"], K)
    b = _dequantize(st["bq"], st["b_scales"], N, K)
    if E == 1:
        return (a @ b[0].t()).to(DTYPES[case["out"]])
    y = torch.bmm(a[st["seg"]], b.transpose(1, 2))
    out = torch.zeros_like(st["out"])
    out[st["live"]] = y[st["has"]].to(out.dtype)
    return out


def _plain_few(st, case):
    T, d, k, dff = case["T"], case["d"], case["k"], case["dff"]
    x = st["x"].float()
    logits = x @ st["router"].t() if case["router"] else st["logits"]
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: lower index
    top, idx = top[:, :k], idx[:, :k].reshape(-1)
    gate = torch.exp(top - top[:, :1])
    gate = gate / gate.sum(dim=1, keepdim=True)
    xk = x.repeat_interleave(k, dim=0).unsqueeze(-1)
    a = _dequantize(st["W1"][0][idx], st["W1"][1][idx], dff, d) @ xk
    b = _dequantize(st["W3"][0][idx], st["W3"][1][idx], dff, d) @ xk
    h = a / (1 + torch.exp(-a)) * b
    y = (_dequantize(st["W2"][0][idx], st["W2"][1][idx], d, dff) @ h).reshape(T, k, d)
    return (gate.unsqueeze(-1) * y).sum(dim=1).to(torch.bfloat16), logits


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        if op == "rows":
            return _plain_quantize(st["x"]).to(st["x"].dtype)
        if op == "weights":
            return _plain_quantize(st["W"].transpose(1, 2)).to(torch.bfloat16)
        if op == "gemm":
            return _plain_gemm(st, case)
        out, logits = _plain_few(st, case)
        return (out, logits) if case["router"] else out

    import combine_fp32_router_gb300 as moe
    if op == "rows":
        q, s = moe.moe_quantize_rows_fp4(st["x"])
        return moe.moe_dequantize_rows_fp4(q, s, case["cols"], st["x"].dtype)
    if op == "weights":
        q, s = moe.moe_quantize_weights_fp4(st["W"])
        return moe.moe_dequantize_rows_fp4(q, s, case["K"], torch.bfloat16)
    if op == "gemm":
        moe.moe_gemm_fp4(st["aq"], st["a_scales"], st["bq"], st["b_scales"], st["out"],
                         case["K"], counts=st.get("counts"))
        return st["out"]
    if "ws" not in st:
        st["ws"] = torch.empty(moe.moe_few_workspace_bytes(case["T"], case["d"], case["E"],
                                                           case["k"], case["dff"]),
                               dtype=torch.uint8, device=DEV)
    moe.moe_forward_few_fp4(st["x"], st["logits"], st["router"] if case["router"] else None,
                            st["W1"][0], st["W3"][0], st["W2"][0], st["W1"][1], st["W3"][1],
                            st["W2"][1], case["k"], st["out"], st["ws"])
    return (st["out"], st["logits"]) if case["router"] else st["out"]


def work(case):
    op = case["op"]
    if op == "rows":
        n, size = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        # values read, codes and scales written and read back, values written
        return dict(bytes=n * (2 * size + 2 * (0.5 + 1 / 32)), flops=4 * n)
    if op == "weights":
        n = case["E"] * case["K"] * case["N"]
        return dict(bytes=n * (4 + 2 * (0.5 + 1 / 32)), flops=4 * n)
    if op == "gemm":
        N, K, rows = case["N"], case["K"], case["rows"]
        size = 4 if case["out"] == "f32" else 2
        hit = sum(c > 0 for c in _shares(case, 1))
        return dict(bytes=(rows + hit * N) * K * (0.5 + 1 / 32) + rows * N * size,
                    flops=2 * rows * N * K)
    T, d, E, k, dff = case["T"], case["d"], case["E"], case["k"], case["dff"]
    hit = E * (1 - (1 - k / E) ** T)  # experts met by T tokens that choose evenly
    route = E * d * 4 if case["router"] else 0
    return dict(bytes=hit * 3 * d * dff * (0.5 + 1 / 32) + 4 * T * d + 4 * T * E + route,
                flops=T * k * 6 * d * dff + (2 * T * E * d if case["router"] else 0))


# ------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The outputs in float64, by table and comparison where the plain form uses arithmetic."""
    st = prepare(case, seed)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    signed = torch.cat([grid, -grid])

    def quantized(rows):  # [R, C] -> what it stands for
        R, C = rows.shape
        out = torch.zeros(R, C, dtype=torch.float64, device=DEV)
        step = max(1, (1 << 24) // C)
        for r in range(0, R, step):
            v = rows[r:r + step].double()
            kp = _up(C, 32)
            v = torch.cat([v, torch.zeros(v.shape[0], kp - C, dtype=v.dtype, device=DEV)], 1)
            v = v.view(v.shape[0], -1, 32)
            top = v.abs().amax(2, keepdim=True)
            e = torch.floor(torch.log2(top.clamp(min=1e-300)))
            e = e - (top < torch.exp2(e)).double() + (top >= torch.exp2(e + 1)).double()
            scale = torch.exp2((e - 2).clamp(-127, 125))
            w = v.abs() / scale
            n = torch.zeros_like(w)  # how many of the eight values lie below
            for i, mid in enumerate((.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0)):
                n += (w >= mid) if i % 2 else (w > mid)
            w = grid[n.long()] * scale * torch.sign(v)
            out[r:r + step] = w.view(w.shape[0], kp)[:, :C]
        return out

    def values(packed, s, rows, K):  # codes [rows, Kp / 2], scale bytes -> [rows, K]
        kp = packed.shape[1] * 2
        code = torch.empty(packed.shape[0], kp, dtype=torch.int64, device=DEV)
        code[:, 0::2] = (packed & 15).long()
        code[:, 1::2] = (packed >> 4).long()
        r = torch.arange(rows, device=DEV)[:, None]
        b = torch.arange(kp // 32, device=DEV)[None, :]
        at = ((r // 128) * (kp // 128) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
        f = torch.exp2(s[at].double() - 127)
        return (signed[code] * f.repeat_interleave(32, dim=1))[:, :K]

    op = case["op"]
    if op == "rows":
        return quantized(st["x"])
    if op == "weights":
        E, K, N = case["E"], case["K"], case["N"]
        return quantized(st["W"].transpose(1, 2).reshape(E * N, K)).view(E, N, K)
    if op == "gemm":
        N, K, E, rows = case["N"], case["K"], case["E"], st["rows"]
        a = values(st["aq"], st["a_scales"], rows, K)
        out = torch.zeros(rows, N, dtype=torch.float64, device=DEV)
        at = 0
        for e, c in enumerate(_shares(case, seed)):
            if c:
                out[at:at + c] = a[at:at + c] @ values(st["bq"][e], st["b_scales"][e], N, K).t()
            at += c if E == 1 else _up(c, 128)
        return out
    T, d, k, dff = case["T"], case["d"], case["k"], case["dff"]
    x = st["x"].double()
    logits = x @ st["router"].double().t() if case["router"] else st["logits"].double()
    out = torch.zeros(T, d, dtype=torch.float64, device=DEV)
    for t in range(T):
        left = logits[t].clone()
        chosen = []
        for _ in range(k):
            j = int((left == left.max()).nonzero()[0])
            chosen.append(j)
            left[j] = -math.inf
        g = torch.softmax(logits[t][chosen], dim=0)
        for j, e in enumerate(chosen):
            a = values(st["W1"][0][e], st["W1"][1][e], dff, d) @ x[t]
            b = values(st["W3"][0][e], st["W3"][1][e], dff, d) @ x[t]
            h = a * torch.sigmoid(a) * b
            out[t] += g[j] * (values(st["W2"][0][e], st["W2"][1][e], d, dff) @ h)
    return (out, logits) if case["router"] else out
