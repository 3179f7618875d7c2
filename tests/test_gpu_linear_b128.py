"""The dense FP8_B128 product (moe_linear_fp8_b128) against the float64 form, elementwise."""
import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def operands(M, N, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    if M > 1:
        x[M // 2] = 0
    # rows and blocks of very different size, so that a scale of the wrong row or block shows
    x *= torch.pow(2.0, torch.randint(-6, 7, (M, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
    w *= torch.pow(2.0, torch.randint(-6, 7, (N, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
    for b in range(0, K, 128):
        x[:, b:b + 128] *= 2.0 ** ((b // 128) % 5 - 2)
    return (*P.quantize_blocks(x), *P.quantize_blocks(w))


def check(out, xq, xs, wq, ws, act):
    xv, wv = P.block_values(xq, xs), P.block_values(wq, ws)
    z = xv @ wv.T
    mag = xv.abs() @ wv.abs().T
    dz = (P.gamma(xv.shape[1]) + 2.0 ** -21) * mag       # the sums, and the scales' three roundings
    if act:
        ref = z.clamp_min(0).square()
        dz = torch.where(z + dz > 0, 2 * z.abs() * dz + dz * dz, torch.zeros_like(z)) + 2.0 ** -23 * ref
    else:
        ref = z
    bound = dz + P.HALF_BF16 * (ref.abs() + dz)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), (int((~(err <= bound)).sum()), float((err / bound.clamp_min(1e-300)).max()))


@pytest.mark.parametrize("M,N,K,act", [
    (1, 16, 16, None), (1, 1856, 2688, "relu2"), (2, 144, 128, None), (7, 272, 208, None), (8, 2688, 1856, None),
    (9, 2688, 1856, "relu2"), (16, 4752, 640, None), (16, 9488, 272, None), (5, 64, 8208, None),
    (17, 16, 16, None), (17, 2688, 1856, None), (64, 2688, 1856, "relu2"), (65, 48, 4112, None), (128, 1856, 2688, None),
    (129, 272, 400, "relu2"), (300, 5136, 272, None), (577, 2688, 1856, None), (1000, 7424, 144, None),
    (2049, 2704, 528, "relu2")])
def test_product(moe, M, N, K, act):
    xq, xs, wq, ws = operands(M, N, K, M * 31 + N * 7 + K)
    out = torch.full((M, N), 3.0, device="cuda", dtype=torch.bfloat16)
    moe.linear_fp8_b128(xq, xs, wq, ws, out, act=act)
    moe.check_device_error()
    check(out, xq, xs, wq, ws, act)
    again = torch.empty_like(out)
    moe.linear_fp8_b128(xq, xs, wq, ws, again, act=act)
    assert torch.equal(out, again)


def test_rows_behind_the_last_stay(moe):
    """M = 130 (a ragged second tile) and M = 5: the rows after M keep their values."""
    for M in (5, 130):
        xq, xs, wq, ws = operands(M, 208, 272, M)
        buf = torch.full((M + 9, 208), 3.0, device="cuda", dtype=torch.bfloat16)
        moe.linear_fp8_b128(xq, xs, wq, ws, buf[:M])
        check(buf[:M], xq, xs, wq, ws, None)
        assert bool((buf[M:] == 3.0).all())


def test_not_a_number_stays_in_its_row_and_column(moe):
    for M in (4, 40):
        xq, xs, wq, ws = operands(M, 64, 256, M)
        ref = torch.empty(M, 64, device="cuda", dtype=torch.bfloat16)
        moe.linear_fp8_b128(xq, xs, wq, ws, ref, act="relu2")
        xq[1, 3] = 127
        ws[7, 1] = float("nan")
        out = torch.empty_like(ref)
        moe.linear_fp8_b128(xq, xs, wq, ws, out, act="relu2")
        nan = torch.isnan(out)
        want = torch.zeros_like(nan)
        want[1], want[:, 7] = True, True
        assert torch.equal(nan, want)
        assert torch.equal(out[~want], ref[~want])


def test_captured_and_replayed(moe):
    for M in (3, 200):
        xq, xs, wq, ws = operands(M, 272, 384, 5)
        out, ref = (torch.empty(M, 272, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            moe.linear_fp8_b128(xq, xs, wq, ws, out)
        for seed in (6, 7):
            for a, b in zip((xq, xs, wq, ws), operands(M, 272, 384, seed)):
                a.copy_(b)
            graph.replay()
            moe.linear_fp8_b128(xq, xs, wq, ws, ref)
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
            check(out, xq, xs, wq, ws, None)
