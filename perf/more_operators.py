"""Workloads of the operators around 8-bit experts: the norm before the layer, rows and weights
in 8 bits, their product, and tokens sorted by expert and back.

Every workload runs in two ways.  With ``own`` false, ``run`` computes the operator from
elementary torch operations in 32 bits; with ``own`` true it makes the calls a user of the
library makes.  ``exact`` computes the same outputs in 64 bits, written separately.

8-bit format: E4M3 codes (largest value 448) with one fp32 scale per row and 128 columns, or per
128 x 128 block of a weight matrix; scale = max(amax / 448, 2^-126), 1 where all values are zero;
a code is the E4M3 number nearest to value * (1 / scale), ties to the even mantissa.  A row of C
values takes round_up(C, 128) bytes, zeros past C.  Outputs in 8 bits are returned as E4M3 numbers
with their scales beside them.

Sorted rows: expert e's rows (token-slot pairs in ascending order) start at a multiple of 128;
rows between the segments are left as they were.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # -- root-mean-square norm with the residual's addition, in the type and in 8 bits
        # one token of the large layer, as in decoding: latency
        dict(name="norm_token", op="norm", rows=1, cols=7168, dtype="bf16", residual=True, pad=0),
        # a prefill batch of the large layer: bandwidth
        dict(name="norm_prefill", op="norm", rows=16384, cols=7168, dtype="bf16", residual=True,
             pad=0),
        # -- its gradient
        # ragged: an odd row count, a width that ends inside a block, fp32
        dict(name="norm_grad_ragged", op="norm_grad", rows=777, cols=1925, dtype="f32",
             residual=False),
        # a training batch, with the gradient that arrives along the residual
        dict(name="norm_grad_train", op="norm_grad", rows=8192, cols=4096, dtype="bf16",
             residual=True),
        # -- 8-bit rows and weights
        # silu(a) * b of the first product's output for the pairs of a training-size batch, in
        # the sorted layout, for the second product
        dict(name="swiglu_rows", op="swiglu", T=8192, k=8, E=128, cols=2048, dtype="bf16"),
        # expert weights [E, K, N] in 128 x 128 blocks, along K: loading a checkpoint
        dict(name="blocks_mid", op="blocks", E=32, K=2048, N=1024),
        # -- products of 8-bit rows and 8-bit weights
        # one token through a projection of the large layer: weight streaming
        dict(name="gemm_token", op="gemm", rows=1, N=4096, K=7168, E=1, out="bf16"),
        # ragged in every size, fp32 out
        dict(name="gemm_ragged", op="gemm", rows=777, N=1545, K=2700, E=1, out="f32"),
        # gate and up projections of the mid layer's experts, 24576 pairs over 64 experts with
        # unequal shares (some empty)
        dict(name="gemm_experts", op="gemm", rows=24576, N=2048, K=2048, E=64, out="bf16"),
        # a dense projection of a prefill batch: tensor-core rate
        dict(name="gemm_prefill", op="gemm", rows=8192, N=7168, K=7168, E=1, out="bf16"),
        # -- tokens sorted by expert and back
        # eight decoding tokens of the large layer: 8-bit rows out, bf16 rows back with weights
        dict(name="sort_decode", op="sort", T=8, k=8, E=256, d=7168, dtype="bf16", train=False,
             drop=0.0),
        # a training batch: rows out and back and both gradients
        dict(name="sort_train", op="sort", T=8192, k=8, E=128, d=4096, dtype="bf16", train=True,
             drop=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "swiglu", "blocks", "gemm", "gemm",
                     "gemm", "sort", "sort", "sort"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    wide = 2 if dtype == "f32" else 1
    if op == "norm":
        cols = _log_int(rng, 33, 8192)
        rows = _log_int(rng, 1, min(65536, 16384 * 7168 // cols // wide))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.6,
                    pad=rng.choice([0, 0, 1, 24]))
    if op == "norm_grad":
        cols = _log_int(rng, 33, 8192)
        rows = _log_int(rng, 1, min(32768, 8192 * 4096 // cols // wide))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.5)
    if op == "swiglu":
        k, E = rng.randint(1, 8), _log_int(rng, 8, 256)
        cols = _log_int(rng, 33, 4096)
        T = _log_int(rng, 1, max(1, min(16384, 8192 * 8 * 2048 // (k * cols * wide) - 16 * E)))
        return dict(op=op, T=T, k=k, E=E, cols=cols, dtype=dtype)
    if op == "blocks":
        K, N = _log_int(rng, 33, 5120), _log_int(rng, 33, 2560)
        return dict(op=op, E=rng.randint(1, max(1, min(64, (64 << 20) // (K * N)))), K=K, N=N)
    if op == "gemm":
        N, K = _log_int(rng, 64, 7168), _log_int(rng, 64, 7168)
        if rng.random() < 0.4:
            E = rng.randint(2, 64)
            rows = _log_int(rng, 1, 24576)
            while E * N * K > 64 * 2048 * 2048 or rows * N * K > 24576 * 2048 * 2048:
                rows, N, K = max(1, rows // 2), max(64, N * 2 // 3), max(64, K * 2 // 3)
        else:
            E = 1
            rows = _log_int(rng, 1, 8192)
        return dict(op=op, rows=rows, N=N, K=K, E=E, out=rng.choice(["bf16", "bf16", "f32"]))
    train = rng.random() < 0.5
    E, k = _log_int(rng, 8, 256), rng.randint(1, 8)
    d = _log_int(rng, 33, 7168)
    T = _log_int(rng, 1, max(1, min(16384, 8192 * 8 * 4096 // (k * d * wide) - 16 * E)))
    return dict(op=op, T=T, k=k, E=E, d=d, dtype=dtype, train=train,
                drop=rng.choice([0.0, 0.0, 0.1]))


def _up(n, m):
    return -(-n // m) * m


def _bound(T, k, E):
    """Rows that sorted pairs can take."""
    return _up(T * k + 127 * min(E, T * k), 128)


# ------------------------------------------------------------------------- the plain format
def _scale(amax):
    s = torch.clamp(amax / 448.0, min=2.0 ** -126)
    return torch.where(amax > 0, s, torch.ones_like(s))


def _quantize(y):
    """E4M3 numbers [R, Kp] and scales [R, Kp / 128] of y [R, C] fp32."""
    R, C = y.shape
    kp = _up(C, 128)
    if kp != C:
        y = torch.nn.functional.pad(y, (0, kp - C))
    y = y.reshape(R, kp // 128, 128)
    s = _scale(y.abs().amax(dim=-1))
    q = (y * (1.0 / s).unsqueeze(-1)).clamp(-448.0, 448.0).to(F8)
    return q.reshape(R, kp), s


def _quantize_blocks(w):
    """E4M3 numbers [E, N, Kp] and scales [E, ceil(N / 128), Kp / 128] of w [E, N, K] fp32."""
    E, N, K = w.shape
    n, k = _up(N, 128), _up(K, 128)
    if (n, k) != (N, K):
        w = torch.nn.functional.pad(w, (0, k - K, 0, n - N))
    w = w.reshape(E, n // 128, 128, k // 128, 128)
    s = _scale(w.abs().amax(dim=(2, 4)))
    q = (w * (1.0 / s)[:, :, None, :, None]).clamp(-448.0, 448.0).to(F8)
    return q.reshape(E, n, k)[:, :N].contiguous(), s


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


def _norm_weight(g, cols, dtype):
    return (1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)).to(dtype)


def _weights8(g, E, N, K):
    """Weights ~ N(0, 1/sqrt(K)) as E4M3 numbers [E, N, Kp] and block scales."""
    kp, per = _up(K, 128), max(1, (1 << 28) // (_up(N, 128) * _up(K, 128)))
    q = torch.empty(E, N, kp, dtype=F8, device=DEV)
    s = torch.empty(E, _up(N, 128) // 128, kp // 128, device=DEV)
    for e in range(0, E, per):
        n = min(per, E - e)
        q[e:e + n], s[e:e + n] = _quantize_blocks(
            torch.randn(n, N, K, generator=g, device=DEV) * K ** -0.5)
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


def _topk(g, case):
    """Experts [T, k] of each token: distinct where E >= k, the low ones more often; a share
    ``drop`` of them -1 (a pair that another rank owns)."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, generator=g, device=DEV)
    logits -= 0.3 * torch.log(1.0 + torch.arange(E, device=DEV))
    idx = torch.topk(logits, min(k, E), dim=1).indices.to(torch.int32)
    if case.get("drop"):
        lost = torch.rand(idx.shape, generator=g, device=DEV) < case["drop"]
        idx = torch.where(lost, torch.full_like(idx, -1), idx)
    return idx.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("norm", "norm_grad"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        st["w"] = _norm_weight(g, cols, dt)
        if op == "norm":
            # pad > 0: rows with a stride, not contiguous
            st["x"] = _activations(g, rows, cols + case["pad"]).to(dt)[:, :cols]
            st["res"] = _activations(g, rows, cols).to(dt) if case["residual"] else None
            st["sum"] = torch.empty(rows, cols, dtype=dt, device=DEV)
            st["out"] = torch.empty(rows, cols, dtype=dt, device=DEV)
            st["q"] = torch.empty(rows, _up(cols, 128), dtype=F8, device=DEV)
            st["scales"] = torch.empty(rows, _up(cols, 128) // 128, device=DEV)
        else:
            st["s"] = _activations(g, rows, cols).to(dt)
            st["rstd"] = torch.rsqrt(st["s"].double().square().mean(dim=1) + EPS).float()
            st["dy"] = torch.randn(rows, cols, generator=g, device=DEV).to(dt)
            st["dsum"] = torch.randn(rows, cols, generator=g, device=DEV).to(dt) \
                if case["residual"] else None
            st["dx"] = torch.empty(rows, cols, dtype=dt, device=DEV)
            st["dw"] = torch.empty(cols, device=DEV)
    elif op == "swiglu":
        # the first product's output for sorted pairs, and which rows hold one
        idx = _topk(g, dict(case, drop=0.0))
        rows, cols, dt = _bound(case["T"], idx.shape[1], case["E"]), case["cols"], \
            DTYPES[case["dtype"]]
        st["ab"] = torch.randn(rows, 2 * cols, generator=g, device=DEV).to(dt)
        perm = _plain_order(idx, case["E"])[1]
        st["perm"], st["live"] = perm, (perm >= 0).nonzero().squeeze(1)
        st["q"] = torch.zeros(rows, _up(cols, 128), dtype=torch.uint8, device=DEV).view(F8)
        st["scales"] = torch.zeros(rows, _up(cols, 128) // 128, device=DEV)
    elif op == "blocks":
        E, K, N = case["E"], case["K"], case["N"]
        st["W"] = (torch.randn(E, K, N, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
    elif op == "gemm":
        E, N, K = case["E"], case["N"], case["K"]
        counts = _shares(case, seed)
        # a buffer that holds the experts' segments, each from a multiple of 128 rows on,
        # however the rows fall
        rows = case["rows"] if E == 1 else _up(case["rows"], 128) + 128 * E
        st["aq"], st["a_scales"] = _quantize(_activations(g, rows, K))
        st["bq"], st["b_scales"] = _weights8(g, E, N, K)
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
        T, E, d, dt = case["T"], case["E"], case["d"], DTYPES[case["dtype"]]
        st["idx"] = _topk(g, case)
        k = st["idx"].shape[1]
        P = _bound(T, k, E)
        gate = torch.rand(T, k, generator=g, device=DEV) + 0.05
        st["gate"] = gate / gate.sum(dim=1, keepdim=True)
        x = _activations(g, T, d)
        if case["train"]:
            st["x"], st["xs"] = x.to(dt), None
            st["rows"] = torch.zeros(P, d, dtype=dt, device=DEV)
            st["dout"] = torch.randn(T, d, generator=g, device=DEV).to(dt)
            st["drows"] = torch.zeros(P, d, dtype=dt, device=DEV)
            st["dgate"] = torch.empty(T, k, device=DEV)
            st["up"] = torch.randn(P, d, generator=g, device=DEV).to(dt)  # d/d sorted rows
            st["dx"] = torch.empty(T, d, dtype=dt, device=DEV)
        else:
            st["x"], st["xs"] = _quantize(x)
            st["rows"] = torch.zeros(P, _up(d, 128), dtype=torch.uint8, device=DEV).view(F8)
            st["rows_s"] = torch.zeros(P, _up(d, 128) // 128, device=DEV)
        st["y"] = torch.randn(P, d, generator=g, device=DEV).to(dt)  # what the experts gave
        st["out"] = torch.empty(T, d, dtype=dt, device=DEV)
        st["counts"] = torch.empty(E, dtype=torch.int32, device=DEV)
        st["perm"] = torch.empty(P, dtype=torch.int32, device=DEV)
        st["pos"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    return st


# ------------------------------------------------------------------------- one pass
def _plain_norm(st, case):
    dt = st["x"].dtype
    s = st["x"].float()
    if st["res"] is not None:
        s = (s + st["res"].float()).to(dt).float()
    rstd = 1.0 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + EPS)
    y = s * rstd * st["w"].float()
    q, scales = _quantize(y)
    got = [y.to(dt), q, scales]
    return got + [s.to(dt)] if st["res"] is not None else got


def _plain_norm_grad(st, case):
    s, dy, r = st["s"].float(), st["dy"].float(), st["rstd"].unsqueeze(1)
    n = s * r
    g = dy * st["w"].float()
    dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return dx.to(st["s"].dtype), (dy * n).sum(dim=0)


def _plain_order(idx, E):
    """counts [E], perm [rows] and pos [T, k] of the experts idx [T, k]."""
    T, k = idx.shape
    e = idx.reshape(-1).long()
    e = torch.where((e >= 0) & (e < E), e, torch.full_like(e, E))
    sorted_e, order = torch.sort(e, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=DEV)
    counts.scatter_add_(0, e, torch.ones_like(e))
    first = torch.cumsum((counts[:E] + 127) // 128 * 128, 0) - (counts[:E] + 127) // 128 * 128
    before = torch.cumsum(counts, 0) - counts
    rank = torch.arange(T * k, device=DEV) - before[sorted_e]
    kept = sorted_e < E
    row = torch.where(kept, first[sorted_e.clamp(max=E - 1)] + rank, torch.full_like(rank, -1))
    pos = torch.empty(T * k, dtype=torch.int32, device=DEV)
    pos[order] = row.to(torch.int32)
    perm = torch.full((_bound(T, k, E) + 1,), -1, dtype=torch.int32, device=DEV)
    perm[torch.where(kept, row, torch.full_like(row, perm.numel() - 1))] = \
        torch.where(kept, order, torch.full_like(order, -1)).to(torch.int32)
    return counts[:E].to(torch.int32), perm[:-1], pos.view(T, k)


def _at(pos, rows):
    """rows[pos] [T, k, d] fp32, zeros where a pair has no row."""
    return rows[pos.clamp(min=0).long()].float() * (pos >= 0).unsqueeze(-1)


def _plain_sort(st, case):
    k = st["idx"].shape[1]
    counts, perm, pos = _plain_order(st["idx"], case["E"])
    got = dict(counts=counts, perm=perm, pos=pos)
    live = perm >= 0
    token = perm.clamp(min=0).long() // k
    raw = st["x"].view(torch.uint8) if st["x"].dtype == F8 else st["x"]
    rows = torch.where(live.unsqueeze(1), raw[token], torch.zeros((), dtype=raw.dtype, device=DEV))
    got["rows"] = rows.view(F8) if st["x"].dtype == F8 else rows
    if st["xs"] is not None:
        got["scales"] = st["xs"][token] * live.unsqueeze(1)
    dt = DTYPES[case["dtype"]]
    y = _at(pos, st["y"])
    got["out"] = (st["gate"].unsqueeze(-1) * y).sum(dim=1).to(dt)
    if case["train"]:
        got["dx"] = _at(pos, st["up"]).sum(dim=1).to(dt)
        dout = st["dout"].float()
        got["dgate"] = (y * dout.unsqueeze(1)).sum(dim=-1)
        g = st["gate"].reshape(-1)[perm.clamp(min=0).long()] * live
        got["drows"] = (g.unsqueeze(1) * dout[token]).to(dt)
    return got


def _plain_gemm(st, case):
    N, K, E = case["N"], case["K"], case["E"]
    kt = st["a_scales"].shape[1]
    a = st["aq"].float().reshape(-1, kt, 128) * st["a_scales"].unsqueeze(-1)
    a = a.reshape(-1, 128 * kt)
    b = st["bq"].float().reshape(E, N, kt, 128)
    b = b * st["b_scales"].repeat_interleave(128, dim=1)[:, :N].unsqueeze(-1)
    b = b.reshape(E, N, 128 * kt)
    if E == 1:
        return (a @ b[0].t()).to(DTYPES[case["out"]])
    y = torch.bmm(a[st["seg"]], b.transpose(1, 2))
    out = torch.zeros_like(st["out"])
    out[st["live"]] = y[st["has"]].to(out.dtype)
    return out


def _plain_swiglu(st, case):
    C = case["cols"]
    ab = st["ab"][st["live"]].float()
    a, b = ab[:, :C], ab[:, C:]
    q, s = _quantize(a / (1.0 + torch.exp(-a)) * b)
    codes = torch.zeros(st["q"].shape, dtype=torch.uint8, device=DEV)
    codes[st["live"]] = q.view(torch.uint8)
    scales = torch.zeros_like(st["scales"])
    scales[st["live"]] = s
    return codes.view(F8), scales


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        if op == "norm":
            return _plain_norm(st, case)
        if op == "norm_grad":
            return _plain_norm_grad(st, case)
        if op == "swiglu":
            return _plain_swiglu(st, case)
        if op == "blocks":
            return _quantize_blocks(st["W"].float().transpose(1, 2))
        if op == "gemm":
            return _plain_gemm(st, case)
        return _plain_sort(st, case)

    import combine_fp32_router_gb300 as moe
    if op == "norm":
        s = st["sum"] if st["res"] is not None else None
        moe.moe_rmsnorm(st["x"], st["w"], EPS, residual=st["res"], sum_out=s, out=st["out"],
                        q=st["q"], scales=st["scales"])
        got = [st["out"], st["q"], st["scales"]]
        return got + [s] if s is not None else got
    if op == "norm_grad":
        if "ws" not in st:
            st["ws"] = torch.empty(moe.moe_rmsnorm_workspace_bytes(case["rows"], case["cols"]),
                                   dtype=torch.uint8, device=DEV)
        moe.moe_rmsnorm_backward(st["dy"], st["s"], st["w"], st["rstd"], st["dx"], st["dw"],
                                 st["ws"], dsum=st["dsum"])
        return st["dx"], st["dw"]
    if op == "swiglu":
        moe.moe_quantize_rows_fp8(st["ab"], q=st["q"], scales=st["scales"], swiglu=True,
                                  perm=st["perm"])
        return st["q"], st["scales"]
    if op == "blocks":
        q, s = moe.moe_quantize_blocks_fp8(st["W"])
        return q.view(F8), s
    if op == "gemm":
        moe.moe_gemm_fp8(st["aq"], st["a_scales"], st["bq"], st["b_scales"], st["out"],
                         case["K"], counts=st.get("counts"))
        return st["out"]
    if "ws" not in st:
        st["ws"] = torch.empty(moe.moe_sort_workspace_bytes(case["T"], case["E"],
                                                            st["idx"].shape[1]),
                               dtype=torch.uint8, device=DEV)
    moe.moe_sort_tokens(st["x"], st["idx"], st["rows"], st["counts"], st["perm"], st["pos"],
                        st["ws"], x_scales=st["xs"], rows_scales=st.get("rows_s"))
    moe.moe_unsort_tokens(st["y"], st["gate"], st["pos"], st["out"], st["ws"])
    got = dict(counts=st["counts"], perm=st["perm"], pos=st["pos"], rows=st["rows"], out=st["out"])
    if st["xs"] is not None:
        got["scales"] = st["rows_s"]
    if case["train"]:
        moe.moe_sort_tokens_backward(st["up"], st["pos"], st["dx"], st["ws"])
        moe.moe_unsort_tokens_backward(st["dout"], st["y"], st["gate"], st["pos"], st["drows"],
                                       st["dgate"], st["ws"])
        got.update(dx=st["dx"], dgate=st["dgate"], drows=st["drows"])
    return got


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, size = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        if op == "norm":  # x and the residual read; their sum, the norm and its 8-bit form written
            return dict(bytes=n * ((4 if case["residual"] else 2) * size + 1 + 4 / 128), flops=8 * n)
        return dict(bytes=n * (4 if case["residual"] else 3) * size, flops=10 * n)
    if op == "swiglu":
        n = case["T"] * min(case["k"], case["E"]) * case["cols"]
        return dict(bytes=n * ((8 if case["dtype"] == "f32" else 4) + 1 + 4 / 128), flops=8 * n)
    if op == "blocks":
        n = case["E"] * case["K"] * case["N"]
        return dict(bytes=n * 3, flops=4 * n)
    if op == "gemm":
        N, K, rows = case["N"], case["K"], case["rows"]
        size = 4 if case["out"] == "f32" else 2
        hit = sum(c > 0 for c in _shares(case, 1))
        return dict(bytes=(rows + hit * N) * K + rows * N * size, flops=2 * rows * N * K)
    T, k, d = case["T"], min(case["k"], case["E"]), case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    pairs = T * k * (1 - case["drop"])
    if not case["train"]:  # 8-bit rows read and written once a pair, the experts' rows read
        return dict(bytes=(T + pairs) * d * (1 + 4 / 128) + (pairs + T) * d * size,
                    flops=2 * pairs * d)
    # out: x, rows; back: y, out; gradients: up, dx; dout, y, drows
    return dict(bytes=d * size * ((T + pairs) * 3 + (T + 2 * pairs)), flops=7 * pairs * d)


# ------------------------------------------------------------------------- 64 bits
def _nearest(v):
    """The E4M3 numbers nearest to v (float64), ties to the even mantissa, by comparison."""
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                        [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    a = v.abs()
    lo = torch.searchsorted(mid, a, right=False)  # midpoints below a
    hi = torch.searchsorted(mid, a, right=True)  # ... and up to a: a tie where they differ
    return grid[torch.where(lo % 2 == 0, lo, hi)] * torch.sign(v)


def _exact_rows(y):
    """(E4M3 numbers, scales) in float64 of y [R, C] float64."""
    R, C = y.shape
    kt = _up(C, 128) // 128
    q = torch.zeros(R, 128 * kt, dtype=torch.float64, device=DEV)
    s = torch.ones(R, kt, dtype=torch.float64, device=DEV)
    for b in range(kt):
        v = y[:, 128 * b:128 * b + 128]
        top = v.abs().max(dim=1).values
        f = torch.where(top > 0, torch.clamp(top / 448, min=2.0 ** -126), torch.ones_like(top))
        s[:, b] = f
        q[:, 128 * b:128 * b + v.shape[1]] = _nearest(v / f[:, None])
    return q, s


def exact(case, seed):
    """The outputs in float64."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        dt = st["x"].dtype
        s = st["x"].double()
        if st["res"] is not None:
            s = (s + st["res"].double()).to(dt).double()
        y = torch.empty_like(s)
        per = max(1, (1 << 25) // case["cols"])
        for r in range(0, case["rows"], per):
            v = s[r:r + per]
            norm = torch.linalg.vector_norm(v, dim=1) / math.sqrt(case["cols"])
            y[r:r + per] = v / torch.hypot(norm, torch.full_like(norm, math.sqrt(EPS)))[:, None]
        y *= st["w"].double()
        q, scales = _exact_rows(y)
        return [y, q, scales, s] if st["res"] is not None else [y, q, scales]
    if op == "norm_grad":
        s, dy, w, r = st["s"].double(), st["dy"].double(), st["w"].double(), st["rstd"].double()
        n = s * r[:, None]
        dot = torch.einsum("rc,rc,c->r", dy, n, w) / case["cols"]
        dx = r[:, None] * (dy * w - n * dot[:, None])
        if st["dsum"] is not None:
            dx += st["dsum"].double()
        return dx, torch.einsum("rc,rc->c", dy, n)
    if op == "swiglu":
        C = case["cols"]
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        s = torch.zeros(st["scales"].shape, dtype=torch.float64, device=DEV)
        for at in torch.split(st["live"], 1 << 14):
            v = st["ab"][at].double()
            q[at], s[at] = _exact_rows(v[:, :C] * torch.sigmoid(v[:, :C]) * v[:, C:])
        return q, s
    if op == "blocks":
        E, K, N = case["E"], case["K"], case["N"]
        kt, nt = _up(K, 128) // 128, _up(N, 128) // 128
        q = torch.zeros(E, N, 128 * kt, dtype=torch.float64, device=DEV)
        s = torch.ones(E, nt, kt, dtype=torch.float64, device=DEV)
        for n in range(nt):
            for k in range(kt):
                v = st["W"][:, 128 * k:128 * k + 128, 128 * n:128 * n + 128].double()
                top = v.abs().reshape(E, -1).max(dim=1).values
                f = torch.where(top > 0, top / 448, torch.ones_like(top))
                s[:, n, k] = f
                q[:, 128 * n:128 * n + v.shape[2], 128 * k:128 * k + v.shape[1]] = \
                    _nearest(v / f[:, None, None]).transpose(1, 2)
        return q, s
    if op == "gemm":
        N, K, E, rows = case["N"], case["K"], case["E"], st["rows"]
        out = torch.zeros(rows, N, dtype=torch.float64, device=DEV)
        at = 0
        for e, c in enumerate(_shares(case, seed)):
            f = st["b_scales"][e].double()
            f = f.repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)
            b = st["bq"][e].double() * f
            a = st["aq"][at:at + c].double()
            a = a * st["a_scales"][at:at + c].double().repeat_interleave(128, dim=1)
            out[at:at + c] = torch.einsum("rk,nk->rn", a, b)
            at += c if E == 1 else _up(c, 128)
        return out
    # ranks by counting the earlier pairs of an expert, one expert at a time
    T, E, d = case["T"], case["E"], case["d"]
    k = st["idx"].shape[1]
    e = st["idx"].reshape(-1).long()
    pos = torch.full((T * k,), -1, dtype=torch.long, device=DEV)
    counts, at = [], 0
    for i in range(E):
        mine = (e == i).nonzero().squeeze(1)
        pos[mine] = at + torch.arange(mine.numel(), device=DEV)
        counts.append(mine.numel())
        at += _up(mine.numel(), 128)
    pair = (pos >= 0).nonzero().squeeze(1)
    row = pos[pair]
    perm = torch.full((_bound(T, k, E),), -1, dtype=torch.long, device=DEV)
    perm[row] = pair
    got = dict(counts=torch.tensor(counts, dtype=torch.int32), perm=perm.to(torch.int32),
               pos=pos.to(torch.int32).view(T, k))
    got["rows"] = torch.zeros(st["rows"].shape, dtype=torch.float64, device=DEV)
    got["rows"][row] = st["x"].double()[pair // k]
    if st["xs"] is not None:
        got["scales"] = torch.zeros(st["rows_s"].shape, dtype=torch.float64, device=DEV)
        got["scales"][row] = st["xs"].double()[pair // k]
    gate = st["gate"].double().reshape(-1)
    got["out"] = torch.zeros(T, d, dtype=torch.float64, device=DEV)
    if case["train"]:
        got["dx"] = torch.zeros(T, d, dtype=torch.float64, device=DEV)
        got["dgate"] = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        got["drows"] = torch.zeros(st["drows"].shape, dtype=torch.float64, device=DEV)
    for j in range(k):  # one slot at a time
        mine = pair[pair % k == j]
        t, r = mine // k, pos[mine]
        y = st["y"][r].double()
        got["out"][t] += gate[mine, None] * y
        if case["train"]:
            got["dx"][t] += st["up"][r].double()
            dout = st["dout"][t].double()
            got["dgate"][mine] = torch.einsum("rd,rd->r", y, dout)
            got["drows"][r] = gate[mine, None] * dout
    if case["train"]:
        got["dgate"] = got["dgate"].view(T, k)
    return got
