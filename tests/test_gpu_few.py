"""The few-token layer (moe_forward_few) against the float64 form, elementwise; indices bit for bit."""
import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


class Layer:
    def __init__(self, moe, T, H, E, K, F, fmt="bf16", ns=0, bias=False, residual=False, seed=0, std=0.05):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def rand(*shape, s=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * s).to(torch.bfloat16)

        self.moe, self.K, self.fmt = moe, K, fmt
        self.x, self.wr = rand(T, H), rand(E, H, s=0.05)
        self.bias = torch.randn(E, generator=g, device="cuda") if bias else None
        self.wu, self.wd = rand(E, F, H, s=std), rand(E, H, F, s=std)
        self.su = self.sd = None
        self.xsc, self.hsc = 4.0 / 448, 12.0 * H * std * std / 448
        if fmt == "e4m3":
            (self.wu, self.su), (self.wd, self.sd) = P.quantize_tensors(self.wu), P.quantize_tensors(self.wd)
        elif fmt == "b128":
            (self.wu, self.su), (self.wd, self.sd) = P.quantize_blocks(self.wu), P.quantize_blocks(self.wd)
        self.shared = (rand(ns * F, H, s=std), rand(H, ns * F, s=std)) if ns else None
        self.res = rand(T, H) if residual else None
        self.d = moe.dims(T, H, E, K, F, fp8=fmt == "e4m3", fp8_b128=fmt == "b128", Fs=ns * F)
        self.sc = None if fmt == "bf16" else moe.fp8_scales(self.su, self.sd, self.xsc, self.hsc)
        self.ws = moe.alloc_workspace(self.d)
        self.ws.fill_(255)
        self.T, self.H = T, H

    def run(self, rows=None, out=None, stream=None):
        x, res, d = self.x, self.res, self.d
        if rows is not None:
            x = x[rows].contiguous()
            res = res[rows].contiguous() if res is not None else None
            d = self.moe.dims(x.shape[0], d.H, d.E, d.K, d.F, fp8=self.fmt == "e4m3", fp8_b128=self.fmt == "b128",
                              Fs=d.Fs)
        T = x.shape[0]
        out = torch.full((T, self.H), 3.0, device="cuda", dtype=torch.bfloat16) if out is None else out
        idx = torch.full((T, self.K), -1, device="cuda", dtype=torch.int32)
        w = torch.full((T, self.K), -1.0, device="cuda")
        self.moe.forward_few(d, x, self.wr, self.bias, self.wu, self.wd, out, self.ws, scales=self.sc, residual=res,
                             topk_idx=idx, topk_w=w, shared=self.shared, stream=stream)
        return out, idx, w

    def reference(self):
        return P.few(self.x, self.wr, self.bias, self.wu, self.wd, self.K, self.fmt, self.su, self.sd, self.xsc,
                     self.hsc, self.shared, self.res)

    def check(self, got=None):
        out, idx, w = got or self.run()
        self.moe.check_device_error()
        ref, bound, ridx, rw = self.reference()
        assert torch.equal(idx, ridx)
        assert float((w.double() - rw).abs().max()) <= 2.0 ** -20
        err = (out.double() - ref).abs()
        assert bool((err <= bound).all()), (int((~(err <= bound)).sum()), float((err / bound).max()))
        return out, idx, w


SIZES = [
    (1, 256, 8, 2, 128), (2, 16, 4, 2, 16), (3, 272, 16, 4, 208), (8, 256, 8, 2, 128), (9, 256, 8, 2, 128),
    (16, 272, 16, 4, 208), (5, 1104, 32, 6, 48), (16, 64, 256, 16, 16), (4, 64, 1, 1, 528), (7, 2688, 12, 6, 1856),
    (2, 4752, 4, 2, 48), (13, 80, 16, 16, 144), (1, 9488, 3, 3, 32), (6, 48, 130, 3, 4112), (11, 304, 40, 8, 1072)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "b128"])
@pytest.mark.parametrize("T,H,E,K,F", SIZES)
def test_layer(moe, T, H, E, K, F, fmt):
    Layer(moe, T, H, E, K, F, fmt, bias=T % 2 == 0, residual=T % 3 != 0, seed=T + H).check()


@pytest.mark.parametrize("T,H,E,K,F,ns", [(1, 256, 8, 2, 128, 1), (7, 272, 16, 4, 208, 2), (16, 1104, 10, 6, 48, 3),
                                          (9, 64, 4, 1, 16, 15), (5, 2688, 9, 6, 1856, 1)])
def test_shared_expert(moe, T, H, E, K, F, ns):
    Layer(moe, T, H, E, K, F, ns=ns, residual=T % 2 == 1, seed=T + H).check()


@pytest.mark.parametrize("cfg", [0, 1])
def test_indices_and_weights_are_the_routers(moe, cfg):
    """Against moe_route at the router's own sizes, ties and near ties among them."""
    L = Layer(moe, 16, 2688, 128, 6, 16, bias=cfg == 1, seed=cfg)
    L.wr[40:45] = L.wr[17]                       # equal logits: the lower index first
    L.wr[100] = L.wr[99]
    L.wr[100, 5] += 0.001953125
    L.x[3] = 0                                   # all logits equal (to the bias)
    _, idx, w = L.run()
    ri, rw = torch.empty_like(idx), torch.empty_like(w)
    moe.route(L.d, L.x, L.wr, L.bias, ri, rw, L.ws)
    moe.check_device_error()
    assert torch.equal(idx, ri)
    assert float((w - rw).abs().max()) <= 1e-5
    if cfg == 0:
        assert idx[3].tolist() == [0, 1, 2, 3, 4, 5]


def test_all_tokens_on_the_same_experts(moe):
    L = Layer(moe, 16, 256, 16, 4, 128, residual=True, seed=3)
    L.x[:] = L.x[0]
    out, idx, _ = L.check()
    assert bool((out - L.res == (out - L.res)).all()) and bool((idx == idx[0]).all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "b128"])
def test_a_token_does_not_depend_on_its_batch(moe, fmt):
    L = Layer(moe, 16, 400, 24, 5, 304, fmt, ns=1 if fmt == "bf16" else 0, residual=True, bias=True, seed=8)
    whole, idx, w = L.run()
    for rows in ([0], [7, 3], list(range(4, 13)), [15, 0, 5, 9, 2]):
        out, i, ww = L.run(rows=torch.tensor(rows, device="cuda"))
        assert torch.equal(out, whole[rows]) and torch.equal(i, idx[rows]) and torch.equal(ww, w[rows])


def test_infinities_of_other_experts_do_not_reach_a_token(moe):
    for T in (6, 14):
        L = Layer(moe, T, 256, 16, 2, 128, seed=11)
        clean, idx, _ = L.run()
        e = int(idx[0, 0])
        L.wu[e, 5, 7], L.wd[e, 9, 3], L.wd[e, 200, 100] = float("inf"), float("nan"), float("-inf")
        out, idx2, _ = L.run()
        assert torch.equal(idx, idx2)
        off = ~(idx == e).any(1)
        assert bool(off.any()) and torch.equal(out[off], clean[off])
        assert not bool(torch.isfinite(out[0]).all())


def test_residual_in_place_and_no_outputs_of_the_routing(moe):
    L = Layer(moe, 5, 272, 16, 4, 208, residual=True, seed=2)
    want, _, _ = L.run()
    x = L.res.clone()
    moe.forward_few(L.d, L.x, L.wr, None, L.wu, L.wd, x, L.ws, residual=x)
    assert torch.equal(x, want)


def test_matches_the_whole_layer_call(moe):
    """moe_forward on the same inputs: the same indices, outputs within its bf16 intermediates."""
    L = Layer(moe, 16, 2688, 32, 6, 1856, residual=True, seed=5, std=0.02)
    out, idx, _ = L.run()
    ref, ri = torch.empty_like(out), torch.empty_like(idx)
    moe.forward(L.d, L.x, L.wr, None, L.wu, L.wd, ref, L.ws, residual=L.res, topk_idx=ri)
    moe.check_device_error()
    assert torch.equal(idx, ri)
    assert float((out.float() - ref.float()).abs().max()) <= 1e-2 * float(ref.float().abs().max())


def test_two_calls_at_once_and_a_replayed_graph(moe):
    a, b = (Layer(moe, 4, 1024, 16, 4, 512, seed=s) for s in (21, 22))
    want_a, want_b = a.run()[0], b.run()[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(torch.empty_like(want_a), torch.empty_like(want_b)) for _ in range(20)]
    for oa, ob in outs:
        with torch.cuda.stream(s1):
            a.run(out=oa)
        with torch.cuda.stream(s2):
            b.run(out=ob)
    torch.cuda.synchronize()
    moe.check_device_error()
    for oa, ob in outs:
        assert torch.equal(oa, want_a) and torch.equal(ob, want_b)
    out = torch.empty_like(want_a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.forward_few(a.d, a.x, a.wr, None, a.wu, a.wd, out, a.ws)
        moe.forward_few(a.d, a.x, a.wr, None, a.wu, a.wd, out, a.ws, residual=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    moe.check_device_error()
    once = torch.empty_like(out)
    moe.forward_few(a.d, a.x, a.wr, None, a.wu, a.wd, once, a.ws, residual=want_a)
    assert torch.equal(out, once)


def test_router_magnitudes_beyond_the_exact_range_are_reported(moe):
    L = Layer(moe, 2, 256, 8, 2, 16, seed=1)
    L.x[1, 0] = 2.0 ** 60
    L.run()
    assert moe.check_device_error_status() == moe.MOE_ERANGE
    L.x[1, 0] = 0
    L.check()


def test_an_expired_wait_returns_a_status_and_leaves_the_next_call_whole(moe):
    L = Layer(moe, 3, 272, 16, 4, 208, seed=4)
    want, _, _ = L.run()
    moe.check_device_error()
    try:
        moe.debug_set(1, 200_000_000)
        moe.debug_set(2, 1)                       # the first up unit never reports
        L.run()
        assert moe.check_device_error_status() == moe.MOE_ETIMEOUT
    finally:
        moe.debug_set(2, 0)
        moe.debug_set(1, 0)
    out, _, _ = L.run()
    moe.check_device_error()
    assert torch.equal(out, want)
