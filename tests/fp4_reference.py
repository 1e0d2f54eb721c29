"""MXFP4 in 64 bits: quantisation by table and comparison, and the values of packed codes."""
import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def up(n, m):
    return -(-n // m) * m


def quantized(x):
    """[R, C] -> float64 values that x stands for after quantisation along its rows."""
    R, C = x.shape
    kp = up(C, 32)
    v = torch.zeros(R, kp, dtype=torch.float64, device=x.device)
    v[:, :C] = x.double()
    v = v.view(R, -1, 32)
    top = v.abs().amax(2, keepdim=True)
    finite = torch.isfinite(v).all(2, keepdim=True)
    t = torch.where(finite, top, torch.ones_like(top)).clamp(min=2.0 ** -200)
    e = torch.floor(torch.log2(t))
    e = e - (t < torch.exp2(e)).double() + (t >= torch.exp2(e + 1)).double()
    scale = torch.exp2((e - 2).clamp(min=-127))
    w = v.abs() / scale
    n = torch.zeros_like(w)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        n += (w >= mid) if i % 2 else (w > mid)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    w = grid[n.long()] * scale * torch.sign(v)
    w = torch.where(finite, w, torch.full_like(w, float("nan")))
    return w.view(R, kp)[:, :C]


def values(q, s, rows, K):
    """Codes [rows, bytes] and tiled scale bytes -> float64 [rows, K]."""
    kp = q.shape[1] * 2
    signed = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64, device=q.device)
    code = torch.empty(q.shape[0], kp, dtype=torch.int64, device=q.device)
    code[:, 0::2] = (q & 15).long()
    code[:, 1::2] = (q >> 4).long()
    r = torch.arange(rows, device=q.device)[:, None]
    b = torch.arange(kp // 32, device=q.device)[None, :]
    at = ((r // 128) * (kp // 128) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
    sb = s.reshape(-1)[at]
    f = torch.where(sb == 255, torch.full(sb.shape, float("nan"), dtype=torch.float64,
                                          device=q.device), torch.exp2(sb.double() - 127))
    return (signed[code[:rows]] * f.repeat_interleave(32, dim=1))[:, :K]


def within(got, want, u):
    """Whether every got is the rounding to its own type of a number within u of want (rounding
    is monotone, so it then lies between the roundings of the two ends)."""
    lo = (want - u).to(torch.float32).to(got.dtype).double()
    hi = (want + u).to(torch.float32).to(got.dtype).double()
    if got.dtype == torch.float32:   # the ends themselves, not rounded inwards
        lo, hi = want - u, want + u
    return bool(((got.double() >= lo) & (got.double() <= hi)).all())


def few(x, logits, W1, W3, W2, k):
    """The layer in float64 on weight values W1, W3 [E, dff, d], W2 [E, d, dff]: the output, and
    a bound on the rounding errors before its last rounding."""
    T, d = x.shape
    x = x.double()
    out = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    err = torch.zeros_like(out)
    eps = 2.0 ** -23
    for t in range(T):
        left = logits[t].double().clone()
        sel = []
        for _ in range(k):
            j = int((left == left.max()).nonzero()[0])
            sel.append(j)
            left[j] = -float("inf")
        g = torch.softmax(logits[t].double()[sel], dim=0)
        for j, e in enumerate(sel):
            a, b = W1[e] @ x[t], W3[e] @ x[t]
            sg = torch.sigmoid(a)
            h = a * sg * b
            # fp32 sums of d terms (relative to the sum of magnitudes, and every partial sum),
            # silu' is at most 1.1; h with 11 significant bits (the six 4-bit terms that carry it
            # keep more than that of all but the smallest values of a block)
            ua = (d + 16) * eps * (W1[e].abs() @ x[t].abs())
            ub = (d + 16) * eps * (W3[e].abs() @ x[t].abs())
            uh = 1.1 * ua * b.abs() + (a * sg).abs() * ub + 16 * eps * h.abs() + 2.0 ** -11 * h.abs()
            # and an absolute floor under the largest
            uh = uh + 2.0 ** -38 * h.abs().amax()
            n = h.numel()
            m = W2[e].abs() @ h.abs()
            out[t] += g[j] * (W2[e] @ h)
            mag[t] += g[j] * m
            err[t] += g[j] * (W2[e].abs() @ uh + (n + 16) * eps * m)
    return out, err + (k + 32) * eps * mag


TERMS = 6                      # MXFP4 numbers that carry an activation of the few-token layer
LEFT = 5.0 ** -TERMS           # of a block's largest value, at most, is what they leave


def block_max(v):
    """Largest magnitude of each value's block of 32 along the last dimension (whole blocks)."""
    return v.abs().view(*v.shape[:-1], -1, 32).amax(-1, keepdim=True).expand(
        *v.shape[:-1], -1, 32).reshape(v.shape)


def in_terms(x, n=TERMS):
    """What n MXFP4 numbers keep of x [.., multiples of 32] (float64): each the nearest to what the
    ones before left, on the smallest power-of-two scale on which none exceeds 6."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    left = x.double().clone()
    for _ in range(n):
        top = block_max(left).clamp(min=2.0 ** -120)
        m, e = torch.frexp(top)                       # top = m 2^e, m in [.5, 1)
        scale = torch.exp2((e - 3 + (m > 0.75)).double())
        w = left.abs() / scale
        k = torch.zeros_like(w, dtype=torch.int64)
        for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
            k += (w >= mid) if i % 2 else (w > mid)
        left = left - grid[k] * scale * torch.sign(left)
    return x.double() - left


def few_in_terms(x, logits, W1, W3, W2, k):
    """few(), with a bound that holds for activations carried as terms: what they leave of x and of
    h is at most LEFT of a block's largest value."""
    T, d = x.shape
    x = x.double()
    out, err = (torch.zeros(T, d, dtype=torch.float64, device=x.device) for _ in range(2))
    eps = 2.0 ** -23
    for t in range(T):
        top, sel = torch.sort(logits[t].double(), descending=True, stable=True)
        g = torch.softmax(top[:k], dim=0)
        ux = LEFT * block_max(x[t])
        mag = torch.zeros_like(out[t])
        for j, e in enumerate(sel[:k].tolist()):
            w1, w3, w2 = W1[e].abs(), W3[e].abs(), W2[e].abs()
            a, b = W1[e] @ x[t], W3[e] @ x[t]
            sg = torch.sigmoid(a)
            h = a * sg * b
            # fp32 sums of TERMS d products, in any order; silu' is at most 1.1
            ua = (TERMS * d + 16) * eps * (w1 @ (x[t].abs() + ux)) + w1 @ ux
            ub = (TERMS * d + 16) * eps * (w3 @ (x[t].abs() + ux)) + w3 @ ux
            uh = 1.1 * ua * (b.abs() + ub) + (a * sg).abs() * ub + 16 * eps * h.abs()
            uh = uh + LEFT * block_max(h.abs() + uh)
            m = w2 @ (h.abs() + uh)
            out[t] += g[j] * (W2[e] @ h)
            err[t] += g[j] * (w2 @ uh + (TERMS * h.numel() + 16) * eps * m)
            mag += g[j] * m
        err[t] += (k + 32) * eps * mag
    return out, err
