"""64-bit references of the training operators, for the tests alone.

Plain definitions (explicit masks, every sum written out), and bounds on what
rounding may do to each result: every stored rounding counts as half a step
of its type (bf16 2^-8 of the value), fp32 arithmetic as 2^-24 an operation.
"""
import numpy as np
import torch

U16 = torch.finfo(torch.bfloat16).eps / 2  # 2^-8
U32 = torch.finfo(torch.float32).eps / 2   # 2^-24


def frame_ids(spans, device="cpu"):
    return torch.repeat_interleave(torch.arange(len(spans), device=device), torch.tensor(list(spans), device=device))


def visible(fi, fj, ref, radius):
    fi, fj = fi[:, None], fj[None, :]
    return (fi < ref) | (fj < ref) | ((fi - fj).abs() <= radius)


def attention(q, k, v, spans, ref, radius):
    """out, lse in 64 bits; q, k, v [H, N, d]."""
    q, k, v = q.double(), k.double(), v.double()
    f = frame_ids(spans, q.device)
    s = (q @ k.transpose(1, 2)) / q.shape[2] ** 0.5
    s = s.masked_fill(~visible(f, f, ref, radius), -np.inf)
    lse = torch.logsumexp(s, 2)
    return torch.exp(s - lse[..., None]) @ v, lse


def attention_backward(q, k, v, out, lse, dout, spans, ref, radius, rows=None):
    """The gradients dq, dk, dv of the rows (all by default) in 64 bits, and
    for each a bound and a standard deviation of its rounding errors.

    The kernel rounds P and dS to bf16 once for the products and each result
    once; everything else is fp32.  Bound: every rounding at its worst, all
    of one sign.  Deviation: roundings independent, each uniform within half
    a step (u / sqrt(3) of the value at most); for dq a common component of
    the keys does not count, because sum_j dS_ij roundings along it are taken
    out again."""
    q, k, v, out, dout, lse = (t.double() for t in (q, k, v, out, dout, lse))
    h, n, d = q.shape
    s = d ** -0.5
    f = frame_ids(spans, q.device)
    rows = torch.arange(n, device=q.device) if rows is None else rows

    def block(qr, kr, fr, fc, q_, k_, v_, do_, o_, lse_):
        # P, dS for query rows x key rows, and the fp32 part of their errors.
        see = visible(fr, fc, ref, radius)
        x = (q_ @ k_.transpose(1, 2)) * s
        p = torch.where(see, torch.exp(x - lse_[..., None]), torch.zeros((), dtype=x.dtype, device=x.device))
        delta = (do_ * o_).sum(2)
        dp = do_ @ v_.transpose(1, 2)
        ds = p * (dp - delta[..., None])
        # exponent: a d-term fp32 product, lse as given, a handful of roundings; 2^-21 for ex2
        ex = (d + 4) * U32 * (q_.abs() @ k_.abs().transpose(1, 2)) * s + 8 * U32 * (x.abs() + lse_.abs()[..., None]) + 2.0 ** -21
        dabs = (d + 8) * U32 * (do_.abs() @ v_.abs().transpose(1, 2) + (do_ * o_).abs().sum(2)[..., None])
        return p, ds, p * ex, ds.abs() * ex + p * dabs

    res = {}
    # dq: the rows against all keys
    p, ds, ep, eds = block(None, None, f[rows], f, q[:, rows], k, v, dout[:, rows], out[:, rows], lse[:, rows])
    dq = s * ds @ k
    m = 8 * U32 * 64  # fp32 accumulation of the products, in 64-row steps
    # With r_j the rounding of dS_ij (|r_j| <= u |dS_ij|) the kernel's dq is s (sum_j (dS_ij + r_j) k_j - (sum_j r_j) c),
    # off by s |sum_j r_j (k_j - c)| <= s u sum_j |dS_ij| (|k_j| + |c|), c the mean key of the first 64 tokens seen.
    at = np.concatenate([[0], np.cumsum(spans)])
    c = torch.zeros(len(spans), h, d, dtype=torch.float64, device=q.device)
    for g in range(len(spans)):
        sees = [x for x in range(len(spans)) if g < ref or x < ref or abs(g - x) <= radius]
        run = next((i for i in range(1, len(sees)) if sees[i] != sees[i - 1] + 1), len(sees))  # the first range's frames
        c[g] = k[:, at[sees[0]]:min(at[sees[0]] + 64, at[sees[run - 1] + 1])].mean(1).abs()
    spread = ds.abs().sum(2, keepdim=True) * c[f[rows]].transpose(0, 1)
    bound = s * ((ds.abs() * (U16 + m) + eds) @ k.abs() + (U16 + m) * spread) * 1.01 + U16 * dq.abs()
    kc = k - k.mean(1, keepdim=True)
    sd = torch.sqrt((s * s * U16 ** 2 / 3) * (ds ** 2 @ kc ** 2) + (U16 * dq) ** 2 / 3 + (s * (eds @ k.abs())) ** 2)
    res["dq"] = (dq, bound, sd)
    # dk, dv: all queries against the rows as keys
    p, ds, ep, eds = block(None, None, f, f[rows], q, k[:, rows], v[:, rows], dout, out, lse)
    pt, dst = p.transpose(1, 2), ds.transpose(1, 2)
    dk, dv = s * dst @ q, pt @ dout
    res["dk"] = (dk, s * ((dst.abs() * (U16 + m) + eds.transpose(1, 2)) @ q.abs()) * 1.1 + U16 * dk.abs(),
                 torch.sqrt((s * s * U16 ** 2 / 3) * (dst ** 2 @ q ** 2) + (U16 * dk) ** 2 / 3 +
                            (s * (eds.transpose(1, 2) @ q.abs())) ** 2))
    res["dv"] = (dv, ((pt * (U16 + m) + ep.transpose(1, 2)) @ dout.abs()) * 1.1 + U16 * dv.abs(),
                 torch.sqrt((U16 ** 2 / 3) * (pt ** 2 @ dout ** 2) + (U16 * dv) ** 2 / 3 +
                            (ep.transpose(1, 2) @ dout.abs()) ** 2))
    return res


def residual_norm(y, x, gamma_post, gamma_pre, gate, frame, alpha, eps):
    """x', h, rstd in 64 bits."""
    y, x = y.double(), x.double()
    g = alpha * gamma_post.double()
    if gate is not None:
        g = g * gate.double()[frame]
    ry = 1 / torch.sqrt((y ** 2).mean(1) + eps)
    xn = x + y * ry[:, None] * g
    rx = 1 / torch.sqrt((xn ** 2).mean(1) + eps)
    return xn, xn * rx[:, None] * gamma_pre.double(), torch.stack([ry, rx])


def residual_norm_backward(dx_out, dh, y, x_out, rstd, gamma_post, gamma_pre, gate, frame, alpha):
    """dx, dy, dgamma_post, dgamma_pre, dgate in 64 bits."""
    dx_out, dh, y, x_out = (t.double() for t in (dx_out, dh, y, x_out))
    ry, rx = rstd.double()[:, :, None]
    yh, xh = y * ry, x_out * rx
    a = dh * gamma_pre.double()
    g = dx_out + rx * (a - xh * (a * xh).mean(1, keepdim=True))
    coef = alpha * (1.0 if gate is None else gate.double()[frame])
    b = coef * g * gamma_post.double()
    dy = ry * (b - yh * (b * yh).mean(1, keepdim=True))
    dgate = None
    if gate is not None:
        dgate = torch.zeros_like(gate, dtype=torch.float64)
        dgate.index_add_(0, frame, alpha * gamma_post.double() * yh * g)
    return g, dy, (coef * yh * g).sum(0), (dh * xh).sum(0), dgate


def e4m3_values():
    """The 256 e4m3 codes' values (bias 7, 3 mantissa bits, 0x7f and 0xff NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    val = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    val[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -val, val)


def checkpoint_pack(x):
    """codes, scales (numpy uint8) of x [..., C] by searching all codes."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    a = np.where(np.isfinite(b), np.abs(b), 0).max(-1)
    scale = np.zeros(a.shape, dtype=np.int64)
    while True:  # the smallest byte whose power of two brings the largest magnitude to at most 448
        low = a > 448 * 2.0 ** (scale - 127.0)
        if not low.any():
            break
        scale[low] += 1
    t = b / 2.0 ** (scale[..., None] - 127.0)
    val = e4m3_values()[:127]  # codes 0 .. 126, increasing
    m = np.abs(np.where(np.isfinite(t), t, 0))
    i = np.clip(np.searchsorted(val, m), 1, 126)  # val[i-1] < m <= val[i]
    lo, hi = m - val[i - 1], val[i] - m
    code = np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)  # ties to the even code
    code = np.where(m == 0, 0, code) | np.where(np.signbit(t), 128, 0)
    code = np.where(np.isfinite(t), code, 127)
    return code.astype(np.uint8).reshape(x.shape), scale.astype(np.uint8)


def checkpoint_unpack(codes, scales):
    v = e4m3_values()[codes].reshape(*codes.shape[:-1], -1, 32)
    return (v * 2.0 ** (scales[..., None].astype(np.float64) - 127)).reshape(codes.shape)
