"""Plain forms of the operators around 8-bit experts, for the tests: the 8-bit format in fp32 (equal
bit for bit) and everything else in float64."""
import torch

U = 2.0 ** -24  # half a step of fp32
F8 = torch.float8_e4m3fn
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def up(n, m=128):
    return -(-n // m) * m


def half_step(dt):
    """The largest relative error of a rounding to dt from fp32 (0 for fp32 itself), and the absolute
    one below its smallest normal."""
    return {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
            torch.float32: (0.0, 2.0 ** -149)}[dt]


def scales_of(amax):
    s = torch.clamp(amax * torch.tensor(1.0 / 448.0, dtype=torch.float32), min=2.0 ** -126)
    s = torch.where(amax > 0, s, torch.ones_like(s))
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))


def codes_of(x, s):
    """uint8 codes of x fp32 with scales s (broadcast): zeros where s is NaN."""
    v = x * (1.0 / s)
    v = torch.where(torch.isnan(s).expand_as(v), torch.zeros_like(v), v)
    return v.clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def quantize_rows(x):
    """codes [R, Kp] uint8 and scales [R, Kp / 128] of x [R, C] fp32."""
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, up(C) - C)).reshape(R, -1, 128)
    amax = b.abs().amax(dim=-1)
    amax = torch.where(torch.isnan(b).any(dim=-1), torch.full_like(amax, float("inf")), amax)
    s = scales_of(amax)
    return codes_of(b, s.unsqueeze(-1)).reshape(R, -1), s


def quantize_blocks(W):
    """codes [E, N, Kp] and scales [E, N / 128, K / 128] of W [E, K, N] fp32."""
    E, K, N = W.shape
    w = torch.nn.functional.pad(W.transpose(1, 2), (0, up(K) - K, 0, up(N) - N))
    w = w.reshape(E, up(N) // 128, 128, up(K) // 128, 128)
    amax = w.abs().amax(dim=(2, 4))
    amax = torch.where(torch.isnan(w).any(dim=4).any(dim=2), torch.full_like(amax, float("inf")), amax)
    s = scales_of(amax)
    q = codes_of(w, s[:, :, None, :, None])
    return q.reshape(E, up(N), up(K))[:, :N].contiguous(), s


def rows64(q, s, C):
    """float64 values of 8-bit rows."""
    v = q.view(F8).to(torch.float64).reshape(q.shape[0], -1, 128) * s.double().unsqueeze(-1)
    return v.reshape(q.shape[0], -1)[:, :C]


def weights64(q, s, K):
    """float64 values [N, K] of one 8-bit matrix with block scales."""
    N = q.shape[0]
    f = s.double().repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)
    return (q.view(F8).to(torch.float64) * f)[:, :K]


def norm64(s, w, eps):
    """(y, rstd) in float64."""
    s = s.double()
    rstd = 1.0 / torch.sqrt(s.square().mean(dim=1) + eps)
    return s * rstd.unsqueeze(1) * w.double(), rstd


def norm_grad64(dy, s, w, rstd, dsum=None):
    """(dx, dw) in float64, and how far fp32 arithmetic with sums of up to 24 steps in a row, and of
    `rows` + 40 steps in dw, may take the results from them."""
    s, dy, w, r = s.double(), dy.double(), w.double(), rstd.double().unsqueeze(1)
    n, g = s * r, dy * w
    m = (g * n).mean(dim=1, keepdim=True)
    dx = r * (g - n * m)
    off = r * U * (4 * g.abs() + n.abs() * (4 * m.abs() + 28 * (g * n).abs().mean(dim=1, keepdim=True)))
    if dsum is not None:
        dx = dx + dsum.double()
        off = off + 2 * U * dx.abs()
    dw = (dy * n).sum(dim=0)
    dw_off = (s.shape[0] + 40) * U * (dy * n).abs().sum(dim=0)
    return dx, dw, off, dw_off


def sort_ref(idx, E, n_rows):
    """counts, perm, pos of experts idx [T, k] (a CPU tensor), one pair after the other."""
    counts = [0] * E
    flat = idx.reshape(-1).tolist()
    for e in flat:
        if 0 <= e < E:
            counts[e] += 1
    first, at = [], 0
    for c in counts:
        first.append(at)
        at += up(c)
    perm, pos = [-1] * n_rows, []
    for p, e in enumerate(flat):
        if 0 <= e < E:
            perm[first[e]] = p
            pos.append(first[e])
            first[e] += 1
        else:
            pos.append(-1)
    i32 = torch.int32
    return torch.tensor(counts, dtype=i32), torch.tensor(perm, dtype=i32), \
        torch.tensor(pos, dtype=i32).view(idx.shape)


def within(got, ref, tol, what):
    """got is within tol of ref, element by element; NaN and infinities in the same places."""
    got, ref = got.double().cpu(), ref.double().cpu()
    tol = tol.double().cpu() if torch.is_tensor(tol) else torch.full_like(ref, float(tol))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got[odd]), torch.isnan(ref[odd])), what
    bad = ((got - ref).abs() > tol) & ~odd | (~torch.isfinite(got) & ~odd)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError("%s: %d of %d values too far off; first at %d: %r for %r (allowed %r)" % (
            what, int(bad.sum()), bad.numel(), i, float(got.reshape(-1)[i]),
            float(ref.reshape(-1)[i]), float(tol.expand_as(ref).reshape(-1)[i])))
