"""The norms between blocks (moe_prenorm, moe_postnorm) against the float64 form, elementwise."""
import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def close(got, ref, bound):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (int(bad.sum()), float((err / bound.clamp_min(1e-300)).max()))


def check_codes(codes, scales, u, du, H):
    """Scales within the bound of the largest value; each code's value within half an E4M3 step of u / scale,
    whatever side of a border its fp32 value fell on; zero codes past H."""
    T, kb = scales.shape
    pad = kb * 128 - H
    uu = torch.nn.functional.pad(u, (0, pad)).view(T, kb, 128)
    dd = torch.nn.functional.pad(du, (0, pad)).view(T, kb, 128)
    amax = uu.abs().amax(-1)
    ref = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    dmax = dd.amax(-1) / 448.0
    close(scales, ref, dmax + 2.0 ** -23 * ref)
    s = scales.double()[..., None]
    got = P.e4m3_value(codes).view(T, kb, 128)
    q, dq = uu / s, dd / s + 2.0 ** -23 * (uu / s).abs()
    lo, hi = P.e4m3_round(q - dq), P.e4m3_round(q + dq)
    assert bool(((got >= lo) & (got <= hi)).all())
    if pad:
        assert int(codes.view(T, kb * 128)[:, H:].max()) == 0


SHAPES = [(1, 16), (1, 2688), (3, 128), (5, 144), (37, 272), (64, 2688), (2, 8192), (3, 12304), (2, 33040), (1, 65536),
          (700, 256), (4097, 48), (1500, 2704)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gain", [True, False])
def test_prenorm(moe, T, H, gain):
    g = gen(T * 7919 + H)
    x = rand(g, T, H, std=3.0)
    if T > 2:
        x[1] = 0                                   # mean 0: u = 0, scale 1
    gv = 1 + rand(g, H, std=0.2) if gain else None
    u = torch.full((T, H), 7.0, device="cuda", dtype=torch.bfloat16)
    kp = moe.b128_kp(H)
    codes = torch.full((T, kp), 255, device="cuda", dtype=torch.uint8)
    scales = torch.full((T, kp // 128), -1.0, device="cuda")
    moe.prenorm(x, gv, u=u, codes=codes, scales=scales, eps=1e-5)
    moe.check_device_error()
    _, _, ref, du = P.norm(x, gv, 1e-5)
    close(u, ref, du + P.HALF_BF16 * (ref.abs() + du))
    check_codes(codes, scales, ref, du, H)
    only = torch.empty_like(u)
    moe.prenorm(x, gv, u=only, eps=1e-5)
    assert torch.equal(only, u)
    c2, s2 = torch.zeros_like(codes), torch.zeros_like(scales)
    moe.prenorm(x, gv, codes=c2, scales=s2, eps=1e-5)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    moe.prenorm(x, gv, u=x, eps=1e-5)              # in place
    assert torch.equal(x, u)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_postnorm(moe, T, H, gate):
    g = gen(T * 104729 + H)
    x, y = rand(g, T, H, std=3.0), rand(g, T, H, std=0.3)
    if T > 2:
        y[2] = 0                                   # an empty block output leaves x
    gp, gn = 1 + rand(g, H, std=0.2), 1 + rand(g, H, std=0.2)
    gv = {"none": None, "channel": rand(g, H), "token": rand(g, T, H)}[gate]
    x_out, u = torch.empty_like(x), torch.empty_like(x)
    kp = moe.b128_kp(H)
    codes = torch.full((T, kp), 255, device="cuda", dtype=torch.uint8)
    scales = torch.full((T, kp // 128), -1.0, device="cuda")
    moe.postnorm(y, gp, x, x_out, gate=gv, alpha=0.7, eps=1e-6, next_gain=gn, u=u, codes=codes, scales=scales)
    moe.check_device_error()
    xp, dx, ref, du = P.norm(x, gn, 1e-6, y=y, gain_post=gp, gate=gv, alpha=0.7)
    close(x_out, xp, dx + P.HALF_BF16 * (xp.abs() + dx))
    close(u, ref, du + P.HALF_BF16 * (ref.abs() + du))
    check_codes(codes, scales, ref, du, H)
    if T > 2:
        assert torch.equal(x_out[2], x[2])
    # the sum alone, without gains, into x itself; u in place of y
    xp, dx, _, _ = P.norm(x, None, 1e-6, y=y, gate=gv, alpha=-1.0)
    x2, y2 = x.clone(), y.clone()
    moe.postnorm(y2, None, x2, x2, gate=gv, alpha=-1.0, eps=1e-6)
    close(x2, xp, dx + P.HALF_BF16 * (xp.abs() + dx))
    x3, y3 = x.clone(), y.clone()
    moe.postnorm(y3, gp, x3, x3, gate=gv, alpha=0.7, eps=1e-6, next_gain=gn, u=y3)
    assert torch.equal(x3, x_out) and torch.equal(y3, u)


def test_norms_are_captured_and_replayed_on_another_stream(moe):
    T, H = 33, 2688
    g = gen(1)
    x, y = rand(g, T, H), rand(g, T, H)
    gp = 1 + rand(g, H, std=0.2)
    x_out, u = torch.empty_like(x), torch.empty_like(x)
    ref_x, ref_u = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.postnorm(y, gp, x, x_out, next_gain=gp, u=u)
    for seed in (2, 3):
        g = gen(seed)
        x.copy_(rand(g, T, H))
        y.copy_(rand(g, T, H))
        graph.replay()
        moe.postnorm(y, gp, x, ref_x, next_gain=gp, u=ref_u)
        torch.cuda.synchronize()
        assert torch.equal(x_out, ref_x) and torch.equal(u, ref_u)


def test_infinities_stay_in_their_row(moe):
    T, H = 4, 256
    g = gen(9)
    x, y = rand(g, T, H), rand(g, T, H)
    clean_x, clean_u = torch.empty_like(x), torch.empty_like(x)
    moe.postnorm(y, None, x, clean_x, u=clean_u)
    y[1, 3], y[2, 5] = float("inf"), float("nan")
    x_out, u = torch.empty_like(x), torch.empty_like(x)
    moe.postnorm(y, None, x, x_out, u=u)
    assert bool(torch.isnan(x_out[1, 3])) and bool(torch.isnan(x_out[2]).all())
    for t in (0, 3):
        assert torch.equal(x_out[t], clean_x[t]) and torch.equal(u[t], clean_u[t])
