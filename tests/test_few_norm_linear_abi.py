"""Refusals of the few-token layer, the norms and the FP8_B128 product, answered on the host before any device
call; and the plain forms' E4M3 helpers against torch's conversion."""
import ctypes

import pytest
import torch

import _plain as P

FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def few(moe, d, scales=None, **kw):
    a = dict(x=FAKE, wr=FAKE, bias=None, wu=FAKE, wd=FAKE, us=None, ds=None, res=None, out=ctypes.c_void_p(8192),
             idx=None, w=None, ws=FAKE, n=1 << 30)
    a.update(kw)
    return moe.raw_library().moe_forward_few(
        ctypes.byref(d), a["x"], a["wr"], a["bias"], a["wu"], a["wd"], a["us"], a["ds"],
        ctypes.byref(scales) if scales else None, a["res"], a["out"], a["idx"], a["w"], a["ws"], a["n"], None)


def test_few_refusals(moe):
    d = lambda T=4, **kw: moe.dims(T, 2688, 128, 6, 1856, **kw)   # noqa: E731
    assert few(moe, d(17)) == moe.MOE_EUNSUPPORTED
    assert few(moe, d(4, nvfp4=True)) == moe.MOE_EUNSUPPORTED
    assert few(moe, moe.dims(4, 2690, 128, 6, 1856)) == moe.MOE_EINVAL
    for k in ("x", "wr", "wu", "wd", "out", "ws"):
        assert few(moe, d(), **{k: None}) == moe.MOE_EINVAL
        assert few(moe, d(), **{k: ODD}) == moe.MOE_EINVAL
    assert few(moe, d(), res=ODD) == moe.MOE_EINVAL
    assert few(moe, d(), out=FAKE) == moe.MOE_EINVAL              # out is x
    assert few(moe, d(), idx=ctypes.c_void_p(4098)) == moe.MOE_EINVAL
    assert few(moe, d(fp8=True)) == moe.MOE_EINVAL                # scales missing
    assert few(moe, d(), us=FAKE) == moe.MOE_EINVAL               # a shared expert without its width
    assert few(moe, d(Fs=1856), us=FAKE) == moe.MOE_EINVAL        # one of its two weights
    assert few(moe, d(fp8=True, Fs=1856)) == moe.MOE_EUNSUPPORTED
    assert few(moe, d(0), x=None, wr=None, wu=None, wd=None, out=None, ws=None, n=0) == moe.MOE_OK


def test_workspace_covers_the_few_token_layer(moe):
    for T, H, E, K, F in [(16, 16, 256, 1, 16), (1, 16, 256, 1, 16), (16, 2688, 128, 6, 1856), (16, 16, 16, 16, 65536)]:
        for kw in ({}, dict(fp8=True), dict(fp8_b128=True)):
            fp8 = bool(kw)
            need = 8 * T * E + (T * H if fp8 else 0) + T * K * F * (1 if fp8 else 4) + 4 * T * K * H
            assert moe.workspace_size(moe.dims(T, H, E, K, F, **kw)) >= need


def test_norm_refusals(moe):
    lib = moe.raw_library()
    pre = lambda T=4, H=256, eps=1e-5, x=FAKE, g=None, u=FAKE, c=None, s=None: lib.moe_prenorm(  # noqa: E731
        T, H, eps, x, g, u, c, s, None)
    assert pre(T=-1) == pre(H=8) == pre(H=264) == pre(H=65552) == moe.MOE_EINVAL
    assert pre(eps=-1.0) == pre(eps=float("nan")) == pre(eps=float("inf")) == moe.MOE_EINVAL
    assert pre(x=None) == pre(u=None) == pre(c=FAKE) == pre(s=FAKE) == moe.MOE_EINVAL
    assert pre(x=ODD) == pre(g=ODD) == pre(u=ODD) == pre(c=ODD, s=FAKE) == pre(c=FAKE, s=ctypes.c_void_p(2)) \
        == moe.MOE_EINVAL
    assert pre(T=0, x=None, u=None) == moe.MOE_OK
    OUT = ctypes.c_void_p(8192)

    def post(T=4, H=256, eps=1e-5, alpha=1.0, y=FAKE, g=None, gate=None, ld=0, x=FAKE, xo=OUT, ng=None, u=None, c=None,
             s=None):
        return lib.moe_postnorm(T, H, eps, alpha, y, g, gate, ld, x, xo, ng, u, c, s, None)

    assert post(H=40) == post(alpha=float("nan")) == post(alpha=float("inf")) == moe.MOE_EINVAL
    assert post(gate=FAKE, ld=128) == post(y=None) == post(x=None) == post(xo=None) == moe.MOE_EINVAL
    assert post(u=OUT) == post(c=FAKE) == moe.MOE_EINVAL          # u is x_out; codes without scales
    for k in ("y", "g", "gate", "x", "xo", "ng", "u"):
        assert post(**{k: ODD}) == moe.MOE_EINVAL
    assert post(T=0, y=None, x=None, xo=None) == moe.MOE_OK


def test_linear_refusals(moe):
    def lin(M=4, N=64, K=128, xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, act=0, out=FAKE):
        return moe.raw_library().moe_linear_fp8_b128(M, N, K, xc, xs, wc, ws, act, out, None)

    assert lin(M=-1) == lin(M=2 ** 31) == lin(N=8) == lin(N=24) == lin(N=2 ** 20 + 16) == moe.MOE_EINVAL
    assert lin(K=8) == lin(K=24) == lin(K=65552) == lin(act=2) == moe.MOE_EINVAL
    for k in ("xc", "xs", "wc", "ws", "out"):
        assert lin(**{k: None}) == moe.MOE_EINVAL
        assert lin(**{k: ctypes.c_void_p(4098)}) == moe.MOE_EINVAL
    assert lin(M=0, xc=None, xs=None, out=None) == moe.MOE_OK


def test_python_arguments_are_checked_before_the_call(moe):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)                 # not a CUDA tensor
    c = torch.zeros(4, 256, dtype=torch.uint8)
    for call in (lambda: moe.linear_fp8_b128(c, torch.zeros(4, 2), c, torch.zeros(4, 2), x),
                 lambda: moe.linear_fp8_b128(c, torch.zeros(4, 2), c, torch.zeros(4, 2), x, act="gelu")):
        with pytest.raises((moe.MoeError, RuntimeError)):
            call()


def test_plain_e4m3_matches_torch():
    v = torch.cat([torch.linspace(-460, 460, 4001), torch.randn(4000) * 2.0 ** -7, torch.tensor([0.0, -0.0])]).double()
    want = v.float().clamp(-448, 448).to(torch.float8_e4m3fn)
    got = P.e4m3_round(v.float().double())
    assert torch.equal(got.float(), want.float())
    assert torch.equal(P.e4m3_codes(got), want.view(torch.uint8))
    codes = torch.arange(256, dtype=torch.uint8)
    val = P.e4m3_value(codes)
    ok = (codes & 127) != 127
    assert torch.equal(val[ok].float(), codes.view(torch.float8_e4m3fn).float()[ok])
