"""Plain float64 forms of the few-token layer, the norms and the FP8_B128 product, with elementwise error
bounds derived from the kernels' arithmetic (torch float64; nothing here calls the library).

Roundings counted: a stored bf16 value is off by at most half a step, 2^-8 of it (E4M3: 2^-4); an fp32 sum of
n terms, in any order and with accumulators that may truncate, by at most n 2^-23 of the sum of magnitudes."""
from __future__ import annotations

import torch

E4M3_MAX = 448.0
HALF_BF16 = 2.0 ** -8


def gamma(n):
    return n * 2.0 ** -23


def e4m3_value(codes):
    """float64 values of E4M3 codes (uint8), from the bit fields."""
    b = codes.to(torch.int32)
    m, e = (b & 7).double(), (b >> 3) & 15
    mag = torch.where(e > 0, (8 + m) * torch.ldexp(torch.ones_like(m), e - 10), m * 2.0 ** -9)
    mag = torch.where((b & 127) == 127, torch.full_like(mag, float("nan")), mag)
    return torch.where(b >= 128, -mag, mag)


def e4m3_round(v):
    """Nearest E4M3 value (float64 in and out), ties to the even code, saturating."""
    a = v.abs()
    e = (torch.frexp(a)[1] - 1).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(a), e - 3)      # exact, unlike a power on the device
    q = ((a / step).round() * step).clamp_max(E4M3_MAX)
    return torch.copysign(q, v)


def e4m3_codes(v):
    """uint8 codes of float64 values that are E4M3 values."""
    table = e4m3_value(torch.arange(256, dtype=torch.uint8, device=v.device))
    pos = table[:127]
    i = torch.searchsorted(pos, v.abs().contiguous())
    return (i + torch.where(torch.signbit(v), 128, 0)).to(torch.uint8)


def quantize_tensors(w):
    """[E, r, c] bf16 -> E4M3 codes with one scale per matrix: codes, scales [E]."""
    amax = w.double().abs().amax((1, 2))
    s = torch.where(amax > 0, (amax.float() / E4M3_MAX), torch.ones_like(amax, dtype=torch.float32))
    return e4m3_codes(e4m3_round((w.float() / s[:, None, None]).double())), s


def quantize_blocks(w):
    """[..., K] bf16 or fp32 -> FP8_B128: codes [..., Kp], scales [..., Kp / 128]."""
    K = w.shape[-1]
    kb = (K + 127) // 128
    v = torch.nn.functional.pad(w.float(), (0, kb * 128 - K)).view(*w.shape[:-1], kb, 128)
    amax = v.abs().amax(-1)
    s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    c = e4m3_codes(e4m3_round((v / s[..., None]).double()))
    return c.view(*w.shape[:-1], kb * 128), s


def block_values(codes, scales):
    kb = scales.shape[-1]
    v = e4m3_value(codes).view(*codes.shape[:-1], kb, 128) * scales.double()[..., None]
    return v.view(codes.shape)


def fixed_logits(x, w_router, bias):
    """[T, E] int64 in units of 2^-40: every product rounded to that grid, summed exactly."""
    p = (x.double()[:, None, :] * w_router.double()[None] * 2.0 ** 40).round().to(torch.int64).sum(-1)
    if bias is not None:
        p = p + (bias.double() * 2.0 ** 40).round().to(torch.int64)
    return p


def few(x, w_router, bias, w_up, w_down, K, fmt="bf16", up_scale=None, down_scale=None, x_scale=1.0, h_scale=1.0,
        shared=None, residual=None):
    """The layer in float64: out, elementwise bound of a kernel's |error|, idx, w."""
    T, H = x.shape
    F = w_up.shape[1]
    logits = fixed_logits(x, w_router, bias)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = order.indices[:, :K]
    top = (order.values[:, :K] - order.values[:, :1]).double() * 2.0 ** -40
    w = torch.softmax(top, 1)
    xa = x.double()
    if fmt != "bf16":
        sx = torch.tensor(x_scale, dtype=torch.float32, device=x.device)
        sh = torch.tensor(h_scale, dtype=torch.float32, device=x.device).double()
        xa = e4m3_round((x.float() / sx).double()) * sx.double()

    def matrices(e):
        if fmt == "bf16":
            return w_up[e].double(), w_down[e].double()
        if fmt == "e4m3":
            return e4m3_value(w_up[e]) * up_scale[e].double(), e4m3_value(w_down[e]) * down_scale[e].double()
        return block_values(w_up[e], up_scale[e])[:, :H], block_values(w_down[e], down_scale[e])[:, :F]

    def expert(up, down, v, quantised):
        """Output of one FFN for the row v and the bound of its error."""
        z = up @ v
        dz = (gamma(H + 8) + 2.0 ** -21) * (up.abs() @ v.abs())   # the sum, and three roundings of scales
        lo = (z.abs() - dz).clamp_min(0) * (z > 0)
        hi = torch.where(z + dz > 0, z.abs() + dz, torch.zeros_like(z))
        h = z.clamp_min(0).square()
        h_lo, h_hi = lo.square(), hi.square()
        if quantised:
            tiny = 1 + 2.0 ** -22   # the square and the quotient round too
            h, h_lo, h_hi = (e4m3_round(q / sh) * sh for q in (h, h_lo / tiny, h_hi * tiny))
        else:
            h_lo, h_hi = h_lo * (1 - 2.0 ** -16) , h_hi * (1 + 2.0 ** -16)   # two bf16 parts
        dh = torch.maximum(h - h_lo, h_hi - h)
        y = down @ h
        dy = down.abs() @ dh + gamma(F + 16) * (down.abs() @ (h + dh))
        return y, dy

    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    for t in range(T):
        for k in range(K):
            up, down = matrices(int(idx[t, k]))
            y, dy = expert(up, down, xa[t], fmt != "bf16")
            out[t] += w[t, k] * y
            bound[t] += w[t, k] * dy
            mag[t] += w[t, k] * y.abs()
        if shared is not None:
            y, dy = expert(shared[0].double(), shared[1].double(), x[t].double(), False)
            out[t] += y
            bound[t] += dy + gamma(8) * y.abs()
            mag[t] += y.abs()
        if residual is not None:
            out[t] += residual[t].double()
            mag[t] += residual[t].double().abs()
    # weights: exp and the quotient, a few fp32 steps; the weighted sum over experts and warps
    bound = bound + gamma(K + 64) * mag
    return out, bound + HALF_BF16 * (out.abs() + bound), idx.int(), w


def norm(x, gain, eps, y=None, gain_post=None, gate=None, alpha=1.0):
    """float64: x' (None without y), u, and the relative bound of their fp32 computation."""
    v = x.double()
    H = v.shape[1]
    xp = None
    dv = torch.zeros_like(v)
    rel = gamma(H / 2 + 16)   # half of the squares' sum's error, and the factors' roundings
    if y is not None:
        n = y.double() / (y.double().square().mean(1, keepdim=True) + eps).sqrt()
        for f in (gain_post, gate):
            if f is not None:
                n = n * f.double()
        al = torch.tensor(alpha, dtype=torch.float32).double().item()
        v = v + al * n
        xp = v
        dv = rel * (al * n).abs() + 2.0 ** -23 * v.abs()
    r = 1.0 / (v.square().mean(1, keepdim=True) + eps).sqrt()
    g = gain.double() if gain is not None else torch.ones(H, dtype=torch.float64, device=x.device)
    u = v * r * g
    # r moves by r^3 sum(v dv) / H
    dr = r ** 3 * (v.abs() * dv).sum(1, keepdim=True) / H
    du = (r * dv + v.abs() * dr) * g.abs() + rel * u.abs()
    return xp, dv, u, du
