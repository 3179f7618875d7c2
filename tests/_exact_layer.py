"""Layers of the few-token kind whose every sum is exact in fp32, so that the output is known bit for bit (torch
float64 on the CPU; nothing here calls the library).

- Activations and weights are small integers, scales powers of two: products and partial sums, in any order, are
  integers (or multiples of a power of two) that 24 bits hold.
- h = relu(z)^2 has at most 16 bits, what the bf16 layer keeps of it; quantised layers round it to E4M3 once.
- The K experts that a token chooses have the same router row, so their weights are 1 / K, K a power of two.
- The residual is minus the rest of the sum, rounded to bf16: what is left is the low bits of the sum, which one
  rounding of h or of an expert's output to 8 bits, or a missing value of K, changes."""
from __future__ import annotations

import torch

import _plain as P


def make(T, H, E, K, F, fmt="bf16", ns=0, seed=0):
    """Inputs (CPU) of T tokens; E is a multiple of K, K a power of two."""
    assert E % K == 0 and K & (K - 1) == 0
    g = torch.Generator().manual_seed(seed)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g).double()

    def signs(density, *shape):
        return ints(0, 1, *shape) * 2 - 1 if density >= 1 else \
            (torch.rand(*shape, generator=g) < density).double() * (ints(0, 1, *shape) * 2 - 1)

    # up sums of a standard deviation of about 40 (h below 2^16), at most of the values of a short K
    up_density = min(1.0, 800.0 / H)
    s = dict(T=T, H=H, E=E, K=K, F=F, fmt=fmt, ns=ns)
    s["x"] = ints(-2, 2, T, H)
    s["wr"] = ints(-2, 2, E // K, H).repeat_interleave(K, 0) / 4
    s["wu"], s["wd"] = signs(up_density, E, F, H), signs(0.5, E, H, F)
    s["shared"] = (signs(up_density, ns * F, H), signs(0.5, H, ns * F)) if ns else None
    s["x_scale"], s["h_scale"] = 0.5, 8.0
    if fmt == "e4m3":
        s["su"], s["sd"] = (2.0 ** ints(-1, 1, E) for _ in range(2))
    elif fmt == "b128":
        kb = lambda n: (n + 127) // 128   # noqa: E731
        s["su"], s["sd"] = 2.0 ** ints(-1, 1, E, F, kb(H)), 2.0 ** ints(-1, 1, E, H, kb(F))
    logits = P.fixed_logits(s["x"], s["wr"], None)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    s["idx"] = order.indices[:, :K]
    assert bool((order.values[:, :K] == order.values[:, :1]).all())
    s["res"] = torch.zeros(T, H, dtype=torch.float64)
    s["res"] = -output(s)[0].bfloat16().double()
    return s


def per_value(scales, n):
    return scales.repeat_interleave(128, -1)[..., :n]


def output(s, plant=None):
    """out in float64 before its rounding, and the largest sum of magnitudes (units of the smallest step)."""
    T, H, K, F, fmt = (s[k] for k in ("T", "H", "K", "F", "fmt"))
    quantised = fmt != "bf16"
    out, big = s["res"].clone(), 0.0

    def ffn(up, down, v, quantised):
        nonlocal big
        if plant == "up_tail":
            up = up.clone()
            up[:, -16:] = 0
        if plant == "down_tail":
            down = down.clone()
            down[:, -16:] = 0
        z = up @ v
        big = max(big, float((up.abs() @ v.abs()).max()) * 8)
        h = z.clamp_min(0).square()
        if quantised:
            h = P.e4m3_round(h / s["h_scale"]) * s["h_scale"]
        else:
            assert float(h.max()) < 2 ** 16
            if plant == "h8":
                h = h.bfloat16().double()
        y = down @ h
        big = max(big, float((down.abs() @ h).max()) * 4)
        return y.bfloat16().double() if plant == "y8" else y

    for t in range(T):
        for e in s["idx"][t].tolist():
            up, down = s["wu"][e], s["wd"][e]
            if fmt == "e4m3":
                up, down = up * s["su"][e], down * s["sd"][e]
            elif fmt == "b128":
                up, down = up * per_value(s["su"][e], H), down * per_value(s["sd"][e], F)
            out[t] += ffn(up, down, s["x"][t], quantised) / K
        if s["shared"] is not None:
            out[t] += ffn(*s["shared"], s["x"][t], False)
    return out, big


# T, H, E, K, F, shared chunks: the decoder's widths, a tail of 16 values of K in either product, one block and many
SIZES = [(1, 256, 8, 2, 128, 1), (3, 272, 16, 4, 208, 0), (7, 2688, 12, 4, 1856, 0), (16, 2688, 8, 1, 1856, 1),
         (1, 9488, 4, 2, 32, 0), (5, 64, 8, 2, 4112, 2), (16, 400, 32, 8, 304, 1), (2, 4752, 4, 2, 48, 0)]
FORMATS = ["bf16", "e4m3", "b128"]


def cases():
    return [(fmt, *size) for size in SIZES for fmt in FORMATS if fmt == "bf16" or not size[5]]
