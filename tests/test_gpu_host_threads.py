"""Calls of several host threads at once, each with a stream, buffers and a workspace of its own.

A kernel's limit of dynamic shared memory belongs to the process.  Sizes that need different amounts are called
in turn, so that a launch that relied on a limit another thread had just lowered would be refused."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def bf16(*shape):
    return torch.randn(*shape, device="cuda").to(torch.bfloat16)


def layer(moe, T, few, fmt="bf16", H=256, E=64, K=6, F=128):
    """A call of the layer and its output."""
    d = moe.dims(T, H, E, K, F, fp8=fmt == "e4m3", fp8_b128=fmt == "b128")
    x, wr, out, ws = bf16(T, H), bf16(E, H), torch.empty(T, H, device="cuda", dtype=torch.bfloat16), moe.alloc_workspace(d)
    scales = su = sd = None
    if fmt == "bf16":
        wu, wd = bf16(E, F, H), bf16(E, H, F)
    else:
        wu, wd = (torch.full(s, 56, device="cuda", dtype=torch.uint8) for s in ((E, F, H), (E, H, F)))   # ones
        su, sd = (torch.ones(E, *(s if fmt == "b128" else ()), device="cuda") for s in ((F, H // 128), (H, F // 128)))
        scales = moe.fp8_scales(su, sd, 1.0, 1.0)
    f = moe.forward_few if few else moe.forward

    def call(s, keep=(su, sd)):
        f(d, x, wr, None, wu, wd, out, ws, scales=scales, stream=s)
    return call, out


def product(moe, M, N, K=256):
    def codes(rows):
        return torch.randint(0, 120, (rows, K), device="cuda", dtype=torch.uint8), torch.ones(rows, K // 128, device="cuda")
    x, w = codes(M), codes(N)
    out = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    return lambda s: moe.linear_fp8_b128(*x, *w, out, stream=s), out


CALLS = {
    "few": lambda moe: [layer(moe, T, True) for T in (1, 16)],
    "few_e4m3": lambda moe: [layer(moe, T, True, "e4m3") for T in (1, 16)],
    "product": lambda moe: [product(moe, 8, 2688), product(moe, 8, 10752)],
    "forward": lambda moe: [layer(moe, T, False, fmt) for T in (4, 300, 1500) for fmt in ("bf16", "e4m3", "b128")],
    "router": lambda moe: [layer(moe, 16, False, H=H, E=E) for H, E in ((256, 64), (2688, 128), (512, 16))],
}


@pytest.mark.parametrize("make", [lambda moe: layer(moe, 3, True), lambda moe: layer(moe, 3, True, "b128"),
                                  lambda moe: product(moe, 3, 144), lambda moe: product(moe, 40, 144),
                                  lambda moe: layer(moe, 3, False)],
                         ids=["few", "few_b128", "product_few", "product", "forward"])
def test_the_first_call_of_a_host_thread(moe, make):
    """A new thread has no CUDA context current before its first runtime call."""
    call, out = make(moe)
    call(None)
    torch.cuda.synchronize()
    want, stream, refused = out.clone(), torch.cuda.current_stream(), []
    out.zero_()
    torch.cuda.synchronize()

    def work():
        try:
            call(stream)
        except moe.MoeError as e:
            refused.append(str(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    assert torch.equal(out, want)


@pytest.mark.parametrize("what,threads,rounds", [(w, 8, 20000) if w == "few" else (w, 4, 8000) for w in CALLS],
                         ids=list(CALLS))
def test_host_threads_do_not_disturb_one_another(moe, what, threads, rounds):
    mine = [CALLS[what](moe) for _ in range(threads)]
    for calls in mine:                       # alone first: what each call has to give
        for call, _ in calls:
            call(None)
    torch.cuda.synchronize()
    moe.check_device_error()
    want = [[out.clone() for _, out in calls] for calls in mine]
    refused, start = [], threading.Barrier(threads)

    def work(t):
        stream = torch.cuda.Stream()
        stream.synchronize()                 # makes the device's context current in this thread
        start.wait()
        for i in range(rounds):
            # the threads are at different calls of their lists
            try:
                mine[t][(i + t) % len(mine[t])][0](stream)
            except moe.MoeError as e:
                refused.append(str(e))
            if i % 50 == 0:
                stream.synchronize()
        stream.synchronize()

    ts = [threading.Thread(target=work, args=(t,)) for t in range(threads)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    moe.check_device_error()
    assert not refused, (len(refused), refused[0])
    for calls, w in zip(mine, want):
        for (_, out), ref in zip(calls, w):
            assert torch.equal(out, ref)
