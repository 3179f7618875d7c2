"""The few-token layer bit for bit, on layers whose sums are exact; and tokens that are equal."""
import pytest
import torch

import _exact_layer as X
import _plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def run(moe, s, residual=True):
    fmt, T, H, E, K, F, ns = (s[k] for k in ("fmt", "T", "H", "E", "K", "F", "ns"))

    def bf16(v):
        got = v.bfloat16()
        assert torch.equal(got.double(), v)
        return got.cuda()

    def codes(v):
        kp = (v.shape[-1] + 127) // 128 * 128 if fmt == "b128" else v.shape[-1]
        return P.e4m3_codes(torch.nn.functional.pad(v, (0, kp - v.shape[-1]))).cuda()

    d = moe.dims(T, H, E, K, F, fp8=fmt == "e4m3", fp8_b128=fmt == "b128", Fs=ns * F)
    if fmt == "bf16":
        wu, wd, sc = bf16(s["wu"]), bf16(s["wd"]), None
    else:
        wu, wd = codes(s["wu"]), codes(s["wd"])
        su, sd = s["su"].float().cuda(), s["sd"].float().cuda()
        sc = moe.fp8_scales(su, sd, s["x_scale"], s["h_scale"])
    out = torch.full((T, H), 7.0, device="cuda", dtype=torch.bfloat16)
    idx = torch.empty(T, K, device="cuda", dtype=torch.int32)
    w = torch.empty(T, K, device="cuda")
    ws = moe.alloc_workspace(d)
    ws.fill_(255)
    moe.forward_few(d, bf16(s["x"]), bf16(s["wr"]), None, wu, wd, out, ws, scales=sc, topk_idx=idx, topk_w=w,
                    residual=bf16(s["res"]) if residual else None,
                    shared=tuple(bf16(v) for v in s["shared"]) if ns else None)
    moe.check_device_error()
    return out, idx, w


@pytest.mark.parametrize("fmt,T,H,E,K,F,ns", X.cases())
def test_every_bit(moe, fmt, T, H, E, K, F, ns):
    s = X.make(T, H, E, K, F, fmt, ns, seed=T + H)
    out, idx, w = run(moe, s)
    assert torch.equal(idx.cpu().long(), s["idx"]) and bool((w == 1.0 / K).all())
    want = X.output(s)[0].bfloat16()
    wrong = out.cpu() != want
    assert not bool(wrong.any()), (int(wrong.sum()), wrong.nonzero()[:4].tolist())


@pytest.mark.parametrize("fmt", X.FORMATS)
def test_equal_tokens_get_equal_outputs(moe, fmt):
    s = X.make(16, 400, 32, 4, 304, fmt, seed=5)
    s["x"][:] = s["x"][3]
    out, idx, _ = run(moe, s, residual=False)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(idx, idx[:1].expand_as(idx))
    assert float(out.abs().max()) > 0
