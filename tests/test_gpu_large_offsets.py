"""Offsets past 31 and 32 bits in the few-token layer, the norms and the FP8_B128 product, and the norms' forms
for many wide rows."""
import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


@pytest.mark.parametrize("T,H", [(444, 1040), (500, 4080), (450, 8192), (447, 12304), (444, 16384)])
def test_many_wide_rows(moe, T, H):
    g = gen(H)
    y, x, gate = rand(g, T, H, std=4.0), rand(g, T, H), rand(g, T, H)
    gp, gn = 1 + rand(g, H, std=0.2), 1 + rand(g, H, std=0.2)
    kp = moe.b128_kp(H)
    out, u = torch.empty_like(x), torch.empty_like(x)
    codes = torch.full((T, kp), 255, device="cuda", dtype=torch.uint8)
    scales = torch.full((T, kp // 128), -1.0, device="cuda")
    moe.postnorm(y, gp, x, out, gate=gate, alpha=0.75, next_gain=gn, u=u, codes=codes, scales=scales)
    xp, dx, ref, du = P.norm(x, gn, 1e-5, y=y, gain_post=gp, gate=gate, alpha=0.75)
    assert bool(((out.double() - xp).abs() <= dx + P.HALF_BF16 * (xp.abs() + dx)).all())
    assert bool(((u.double() - ref).abs() <= du + P.HALF_BF16 * (ref.abs() + du)).all())
    # a code's value: the scale's and the product's roundings move u / scale by 2^-22 of it, a code by half a step
    pad = kp - H
    v = torch.nn.functional.pad(ref, (0, pad)).view(T, -1, 128) / scales.double()[..., None]
    d = torch.nn.functional.pad(du, (0, pad)).view(T, -1, 128) / scales.double()[..., None] + 2.0 ** -22 * v.abs()
    got = P.e4m3_value(codes).view(T, -1, 128)
    assert bool(((got >= P.e4m3_round(v - d)) & (got <= P.e4m3_round(v + d))).all())
    # the same numbers from the prenorm of a stored x'
    u2 = torch.empty_like(u)
    moe.prenorm(out, gn, u=u2)
    _, _, ref2, du2 = P.norm(out, gn, 1e-5)
    assert bool(((u2.double() - ref2).abs() <= du2 + P.HALF_BF16 * (ref2.abs() + du2)).all())
    moe.check_device_error()


def test_norm_of_more_than_2_to_31_values(moe):
    T, H = 33000, 65536
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    g = gen(1)
    x[-3:] = rand(g, 3, H)
    x[:2] = rand(g, 2, H)
    u = torch.empty_like(x)
    moe.prenorm(x, u=u)
    moe.check_device_error()
    for rows in (slice(0, 2), slice(T - 3, T)):
        _, _, ref, du = P.norm(x[rows], None, 1e-5)
        assert bool(((u[rows].double() - ref).abs() <= du + P.HALF_BF16 * (ref.abs() + du)).all())
    assert not bool(u[2:-3].any())


def test_product_of_more_than_2_to_31_outputs(moe):
    M, N, K = 131201, 16400, 144
    g = gen(2)
    xq, xs = P.quantize_blocks(rand(g, 5, K))
    wq, ws = P.quantize_blocks(rand(g, N, K, std=0.05))
    rows = torch.tensor([0, 130943, 131071, 131072, M - 1], device="cuda")
    X = torch.zeros(M, xq.shape[1], device="cuda", dtype=torch.uint8)
    S = torch.ones(M, xs.shape[1], device="cuda")
    X[rows], S[rows] = xq, xs
    out = torch.full((M, N), 3.0, device="cuda", dtype=torch.bfloat16)
    moe.linear_fp8_b128(X, S, wq, ws, out)
    moe.check_device_error()
    xv, wv = P.block_values(xq, xs), P.block_values(wq, ws)
    ref = xv @ wv.T
    dz = (P.gamma(xv.shape[1]) + 2.0 ** -21) * (xv.abs() @ wv.abs().T)
    assert bool(((out[rows].double() - ref).abs() <= dz + P.HALF_BF16 * (ref.abs() + dz)).all())
    assert int((out != 0).any(1).sum()) == 5


def test_layer_of_more_than_2_to_32_bytes_of_weights(moe):
    T, H, E, K, F = 3, 2688, 256, 2, 4112
    g = gen(3)
    x, wr = rand(g, T, H), rand(g, E, H, std=0.05)
    bias = torch.zeros(E, device="cuda")
    bias[[0, 201, 254, 255]] = 100.0   # the choice is among these
    wu = torch.zeros(E, F, H, device="cuda", dtype=torch.bfloat16)
    wd = torch.zeros(E, H, F, device="cuda", dtype=torch.bfloat16)
    for e in (0, 201, 254, 255):
        wu[e], wd[e] = rand(g, F, H, std=0.05), rand(g, H, F, std=0.05)
    d = moe.dims(T, H, E, K, F)
    out = torch.full((T, H), 3.0, device="cuda", dtype=torch.bfloat16)
    idx = torch.empty(T, K, device="cuda", dtype=torch.int32)
    moe.forward_few(d, x, wr, bias, wu, wd, out, moe.alloc_workspace(d), topk_idx=idx)
    moe.check_device_error()
    ref, bound, ridx, _ = P.few(x, wr, bias, wu, wd, K)
    assert torch.equal(idx, ridx) and int(idx.max()) >= 201
    assert bool(((out.double() - ref).abs() <= bound).all())
