"""A stack of routed-MoE layers over one residual stream, through the C ABI.

Each layer l applies, to the residual stream x (bf16, [T, H]):
    u = rmsnorm(x)                      (moe_rmsnorm, unit gain)
    x = x + MoE_l(u)                    (moe_forward with residual = x)
with the expert banks in bf16 or in E4M3 codes with scalar scales (W8A8).
The normalisation before each layer follows the pre-norm blocks of the hybrid
decoder: the audio.cpp model page ("Q4_K, Q3_K and Q2_K expert profiles")
names a normalisation among the model's steps; without one, a stack of
these layers grows without bound.

A layer with gains is a sandwich of norms, and may have a dense shared expert in
FP8_B128 beside the routed ones:
    u  = rms(x) * gain_pre                                       (moe_prenorm)
    s  = relu^2(u w_up^T) w_down^T                               (moe_linear_fp8_b128, twice)
    x  = x + alpha * gate * (rms(MoE_l(u) + s) * gain_post)      (moe_postnorm)
whose last step makes the next layer's u as well.  With few=True, at most
FEW_MAX_TOKENS tokens run through the two-launch layer (moe_forward_few).

Marshalling only: every step runs in the library's kernels.
"""
from __future__ import annotations

import torch

from . import (FEW_MAX_TOKENS, alloc_workspace, b128_kp, dims, forward, forward_few, fp8_scales, linear_fp8_b128,
               postnorm, prenorm, quantize_fp8, quantize_fp8_b128, rmsnorm)


def _b128(w):
    """FP8_B128 codes and scales of w [..., rows, K] (bf16)."""
    K, kp = w.shape[-1], b128_kp(w.shape[-1])
    codes = torch.empty(*w.shape[:-1], kp, dtype=torch.uint8, device=w.device)
    scales = torch.empty(*w.shape[:-1], kp // 128, dtype=torch.float32, device=w.device)
    quantize_fp8_b128(w.view(-1, w.shape[-2], K), codes, scales)
    return codes, scales


class MoeStack:
    def __init__(self, T, H, E, K, F, fp8=True, eps=1e-5, device="cuda", fp8_b128=False, few=False):
        """fp8_b128: expert banks with a scale per 128 weights (then fp8 is not looked at)."""
        if few and T > FEW_MAX_TOKENS:
            raise ValueError(f"few: at most {FEW_MAX_TOKENS} tokens, got {T}")
        self.T, self.H, self.E, self.K, self.F = T, H, E, K, F
        self.fp8 = fp8 and not fp8_b128
        self.fp8_b128 = fp8_b128
        self.moe = forward_few if few else forward
        self.eps = eps
        self.device = torch.device(device)
        self.layers = []
        self.dims = dims(T, H, E, K, F, fp8=self.fp8, fp8_b128=fp8_b128)
        self.ws = alloc_workspace(self.dims, self.device)
        self.u = torch.empty(T, H, dtype=torch.bfloat16, device=self.device)
        self.y = self.s = self.codes = self.scales = None   # a sandwich's buffers, and its shared expert's
        self.hidden = {}                                    # by width: activations, codes, scales
        self.x = [torch.empty(T, H, dtype=torch.bfloat16, device=self.device) for _ in range(2)]

    def add_layer(self, w_router, w_up, w_down, x_scale=None, h_scale=None, bias=None, gain_pre=None, gain_post=None,
                  gate=None, alpha=1.0, shared=None):
        """w_up [E,F,H], w_down [E,H,F] as bf16 masters; quantised here when the stack is W8A8.

        gain_post [H] makes the layer a sandwich, with gain_pre [H] or None (ones), gate [H] or [T, H] or None,
        the residual scale alpha, and shared = (w_up [Fs, H], w_down [H, Fs]) as bf16 masters or None."""
        if gain_post is None and not (gain_pre is None and gate is None and alpha == 1.0 and shared is None):
            raise ValueError("gain_pre, gate, alpha and shared belong to a layer with gain_post")
        layer = {"wr": w_router, "bias": bias}
        if self.fp8:
            cu = torch.empty(w_up.shape, dtype=torch.uint8, device=self.device)
            cd = torch.empty(w_down.shape, dtype=torch.uint8, device=self.device)
            su = torch.empty(self.E, dtype=torch.float32, device=self.device)
            sd = torch.empty(self.E, dtype=torch.float32, device=self.device)
            quantize_fp8(w_up, cu, su)
            quantize_fp8(w_down, cd, sd)
            layer.update(wu=cu, wd=cd, su=su, sd=sd, scales=fp8_scales(su, sd, x_scale, h_scale))
        elif self.fp8_b128:
            (cu, su), (cd, sd) = _b128(w_up), _b128(w_down)
            layer.update(wu=cu, wd=cd, su=su, sd=sd, scales=fp8_scales(su, sd, x_scale, h_scale))
        else:
            layer.update(wu=w_up, wd=w_down, scales=None)
        layer.update(gain_pre=gain_pre, gain_post=gain_post, gate=gate, alpha=alpha, shared=None)
        if gain_post is not None and self.y is None:
            self.y = torch.empty_like(self.u)
        if shared is not None:
            layer["shared"] = (*_b128(shared[0]), *_b128(shared[1]))
            if self.codes is None:
                kp = b128_kp(self.H)
                self.codes = torch.empty(self.T, kp, dtype=torch.uint8, device=self.device)
                self.scales = torch.empty(self.T, kp // 128, dtype=torch.float32, device=self.device)
                self.s = torch.empty_like(self.u)
            fs = shared[0].shape[0]
            if fs not in self.hidden:
                h = torch.empty(self.T, fs, dtype=torch.bfloat16, device=self.device)
                self.hidden[fs] = (h, *_b128(h.zero_()))
        self.layers.append(layer)
        return layer

    def _norm_outputs(self, L):
        """What the norm before this layer writes."""
        return {"u": self.u, **({"codes": self.codes, "scales": self.scales} if L["shared"] else {})}

    def run_layer(self, l, x_in, x_out, topk_idx=None, topk_w=None, normed=False, norm_next=False):
        """normed: the step before made this layer's u.  norm_next: make the next layer's (a sandwich's last step)."""
        L = self.layers[l]
        sandwich = L["gain_post"] is not None
        if not normed:
            if sandwich:
                prenorm(x_in, L["gain_pre"], eps=self.eps, **self._norm_outputs(L))
            else:
                rmsnorm(x_in, self.u, self.eps)
        res, out = (None, self.y) if sandwich else (x_in, x_out)
        if L["shared"]:
            cu, su, cd, sd = L["shared"]
            h, hc, hs = self.hidden[cu.shape[0]]
            linear_fp8_b128(self.codes, self.scales, cu, su, h, act="relu2")
            quantize_fp8_b128(h.view(1, *h.shape), hc, hs)
            linear_fp8_b128(hc, hs, cd, sd, self.s)
            res = self.s
        self.moe(self.dims, self.u, L["wr"], L["bias"], L["wu"], L["wd"], out, self.ws, scales=L["scales"],
                 residual=res, topk_idx=topk_idx, topk_w=topk_w)
        if sandwich:
            N = self.layers[l + 1] if norm_next else None
            postnorm(self.y, L["gain_post"], x_in, x_out, gate=L["gate"], alpha=L["alpha"], eps=self.eps,
                     **({"next_gain": N["gain_pre"], **self._norm_outputs(N)} if norm_next else {}))

    def forward(self, x):
        """Run every layer on x (bf16 [T, H]); returns the final residual stream (an internal buffer)."""
        src, normed = x, False
        for l in range(len(self.layers)):
            dst = self.x[l % 2]
            # one pass over x makes both norms between two sandwiches
            both = l + 1 < len(self.layers) and all(L["gain_post"] is not None for L in self.layers[l:l + 2])
            self.run_layer(l, src, dst, normed=normed, norm_next=both)
            src, normed = dst, both
        return src
