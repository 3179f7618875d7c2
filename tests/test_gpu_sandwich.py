"""The new operators as they run together: sandwich layers of the stack (prenorm, the dense FP8_B128 shared
expert, the routed layer, postnorm), against the calls one by one and against the float64 form."""
import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def build(T, fmt, few, n_layers=3, H=272, E=16, K=4, F=144, Fs=208, seed=0):
    from routed_expert_moe_b200.stack import MoeStack
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T)

    def rand(*shape, s=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    st = MoeStack(T, H, E, K, F, fp8=fmt == "e4m3", fp8_b128=fmt == "b128", few=few)
    raw = []
    for l in range(n_layers):
        shared = (rand(Fs + 16 * l, H, s=0.05), rand(H, Fs + 16 * l, s=0.05)) if l != 1 else None
        kw = dict(gain_pre=1 + rand(H, s=0.2) if l else None, gain_post=1 + rand(H, s=0.2),
                  gate=[rand(T, H), None, rand(H)][l % 3], alpha=0.5 + 0.25 * l, shared=shared)
        w = (rand(E, H, s=0.05), rand(E, F, H, s=0.05), rand(E, H, F, s=0.05))
        st.add_layer(*w, x_scale=4.0 / 448, h_scale=12.0 * H * 0.0025 / 448, **kw)
        raw.append((w, kw))
    return st, rand(T, H), raw


@pytest.mark.parametrize("T,few", [(1, True), (7, True), (16, False), (129, False)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "b128"])
def test_stack_is_its_operators_one_by_one(moe, fmt, T, few):
    st, x, _ = build(T, fmt, few)
    y = st.forward(x).clone()
    e = torch.empty_like
    a, u, yy, s = x.clone(), e(x), e(x), e(x)
    kp = moe.b128_kp(st.H)
    codes = torch.empty(T, kp, device="cuda", dtype=torch.uint8)
    scales = torch.empty(T, kp // 128, device="cuda")
    ws = moe.alloc_workspace(st.dims)
    moe.prenorm(a, st.layers[0]["gain_pre"], u=u, codes=codes, scales=scales)
    for l, L in enumerate(st.layers):
        if L["shared"]:
            cu, su, cd, sd = L["shared"]
            h = torch.empty(T, cu.shape[0], device="cuda", dtype=torch.bfloat16)
            moe.linear_fp8_b128(codes, scales, cu, su, h, act="relu2")
            hc = torch.empty(T, cd.shape[1], device="cuda", dtype=torch.uint8)
            hs = torch.empty(T, cd.shape[1] // 128, device="cuda")
            moe.quantize_fp8_b128(h.view(1, *h.shape), hc, hs)
            moe.linear_fp8_b128(hc, hs, cd, sd, s)
        (moe.forward_few if few else moe.forward)(st.dims, u, L["wr"], None, L["wu"], L["wd"], yy, ws,
                                                  scales=L["scales"], residual=s if L["shared"] else None)
        nxt = st.layers[l + 1]["gain_pre"] if l + 1 < len(st.layers) else None
        moe.postnorm(yy, L["gain_post"], a, a, gate=L["gate"], alpha=L["alpha"], next_gain=nxt, u=u, codes=codes,
                     scales=scales)
    moe.check_device_error()
    assert torch.equal(y, a)


@pytest.mark.parametrize("T,few", [(5, True), (40, False)])
def test_layer_against_float64(moe, T, few):
    """One bf16 sandwich with a shared expert, float64 from the stack's own u, codes and routing on."""
    st, x, raw = build(T, "bf16", few, n_layers=1)
    idx = torch.empty(T, st.K, device="cuda", dtype=torch.int32)
    w = torch.empty(T, st.K, device="cuda")
    out = torch.empty_like(x)
    st.run_layer(0, x, out, topk_idx=idx, topk_w=w)
    moe.check_device_error()
    L, ((wr, wu, wd), kw) = st.layers[0], raw[0]
    _, _, u, du = P.norm(x, None, 1e-5)
    assert bool(((st.u.double() - u).abs() <= du + P.HALF_BF16 * (u.abs() + du)).all())
    # the shared expert from the codes of u: its hidden values are rounded to bf16, then to E4M3 per block
    cu, su, cd, sd = L["shared"]
    z = P.block_values(st.codes, st.scales) @ P.block_values(cu, su).T
    h, hc, hs = st.hidden[cu.shape[0]]
    ref_h = z.clamp_min(0).square()
    dz = (P.gamma(cu.shape[1]) + 2.0 ** -21) * (P.block_values(st.codes, st.scales).abs() @ P.block_values(cu, su).abs().T)
    dh = torch.where(z + dz > 0, 2 * z.abs() * dz + dz * dz, torch.zeros_like(z)) + 2.0 ** -23 * ref_h
    assert bool(((h.double() - ref_h).abs() <= dh + P.HALF_BF16 * (ref_h + dh)).all())
    hv, dv = P.block_values(hc, hs), P.block_values(cd, sd)
    s, mag = hv @ dv.T, hv.abs() @ dv.abs().T
    ds = (P.gamma(hv.shape[1]) + 2.0 ** -21) * mag
    assert bool(((st.s.double() - s).abs() <= ds + P.HALF_BF16 * (s.abs() + ds)).all())
    # the routed experts from the bf16 u, beside the stored s as the residual
    if few:
        ref, bound, ridx, rw = P.few(st.u, wr, None, wu, wd, st.K, residual=st.s)
        assert torch.equal(idx, ridx)
        assert bool(((st.y.double() - ref).abs() <= bound).all())
    xp, dxp, _, _ = P.norm(x, None, 1e-5, y=st.y, gain_post=kw["gain_post"], gate=kw["gate"], alpha=kw["alpha"])
    assert bool(((out.double() - xp).abs() <= dxp + P.HALF_BF16 * (xp.abs() + dxp)).all())


def test_run_is_captured_and_replayed(moe):
    """A whole run in a CUDA graph: new inputs in the same buffer, the results of an eager run."""
    st, x, _ = build(6, "b128", True)
    xs = [x.clone(), x.flip(0).contiguous()]
    want = [st.forward(v).clone() for v in xs]
    inp = xs[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y = st.forward(inp)
    for i in (1, 0, 1):
        inp.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    moe.check_device_error()
