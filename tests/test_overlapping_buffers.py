"""Buffers that overlap without being the same: refused on the host before any device call (no GPU; every call here
is one that has to be refused)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


class Memory:
    """Addresses far from one another (nothing is read there), and some inside another's range."""

    def __init__(self):
        self.next = 1 << 20

    def take(self):
        self.next += 1 << 24
        return self.next


def p(v):
    return None if v is None else ctypes.c_void_p(v)


T, H = 4, 256
ROW, ACT = 2 * H, 2 * T * H


def few(moe, x, out, res=None):
    m = Memory()
    d = moe.dims(T, H, 8, 2, 128)
    return moe.raw_library().moe_forward_few(ctypes.byref(d), p(x), p(m.take()), None, p(m.take()), p(m.take()), None,
                                             None, None, p(res), p(out), None, None, p(m.take()), 1 << 30, None)


@pytest.mark.parametrize("by", [0, 16, ROW, ACT - 16, -16, -ROW, 16 - ACT])
def test_few(moe, by):
    a, b = 1 << 30, 1 << 31
    assert few(moe, x=a, out=a + by) == moe.MOE_EINVAL
    if by:
        assert few(moe, x=b, out=a + by, res=a) == moe.MOE_EINVAL


def norm(moe, post, **kw):
    m = Memory()
    a = dict(x=m.take(), g=m.take(), u=m.take(), c=m.take(), s=m.take())
    if post:
        a.update(y=m.take(), gate=m.take(), ld=H, xo=m.take(), ng=m.take())
    for k, (of, by) in kw.items():
        a[k] = a[of] + by
    lib = moe.raw_library()
    if not post:
        return lib.moe_prenorm(T, H, 1e-5, p(a["x"]), p(a["g"]), p(a["u"]), p(a["c"]), p(a["s"]), None)
    return lib.moe_postnorm(T, H, 1e-5, 1.0, p(a["y"]), p(a["g"]), p(a["gate"]), a["ld"], p(a["x"]), p(a["xo"]),
                            p(a["ng"]), p(a["u"]), p(a["c"]), p(a["s"]), None)


@pytest.mark.parametrize("kw", [
    dict(u=("x", ROW)), dict(u=("x", 16)), dict(x=("u", ROW)), dict(u=("g", 0)), dict(g=("u", ACT - 16)),
    dict(c=("x", 0)), dict(c=("u", 0)), dict(c=("u", ACT - 16)), dict(s=("x", 0)), dict(s=("c", T * H - 4)),
    dict(c=("s", 16)), dict(s=("g", 0))], ids=str)
def test_prenorm(moe, kw):
    assert norm(moe, False, **kw) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", [
    dict(xo=("x", ROW)), dict(xo=("y", 16)), dict(x=("xo", ROW)), dict(u=("xo", 0)), dict(u=("xo", ACT - 16)),
    dict(u=("x", ROW)), dict(u=("y", ROW)), dict(y=("u", ROW)), dict(gate=("xo", ROW)), dict(gate=("u", 16)),
    dict(g=("xo", ROW)), dict(ng=("u", ROW)), dict(ng=("xo", 0)), dict(c=("x", 0)), dict(c=("y", 0)), dict(c=("xo", 0)),
    dict(c=("gate", ACT - 16)), dict(s=("y", 4)), dict(s=("xo", 0)), dict(s=("c", 0))], ids=str)
def test_postnorm(moe, kw):
    assert norm(moe, True, **kw) == moe.MOE_EINVAL


def test_a_gate_of_channels_is_no_row_to_replace(moe):
    m = Memory()
    gate, x, y = m.take(), m.take(), m.take()
    lib = moe.raw_library()
    for xo, u in ((gate, None), (m.take(), gate)):
        assert lib.moe_postnorm(T, H, 1e-5, 1.0, p(y), None, p(gate), 0, p(x), p(xo), None, p(u), None, None,
                                None) == moe.MOE_EINVAL


@pytest.mark.parametrize("of", ["xc", "xs", "wc", "ws"])
def test_product(moe, of):
    M, N, K = 4, 64, 256
    size = dict(xc=M * K, xs=M * K // 32, wc=N * K, ws=N * K // 32)
    for by in (0, size[of] - 16, 16 - 2 * M * N):
        m = Memory()
        a = {k: m.take() for k in size}
        out = a[of] + by
        assert moe.raw_library().moe_linear_fp8_b128(M, N, K, p(a["xc"]), p(a["xs"]), p(a["wc"]), p(a["ws"]), 0, p(out),
                                                     None) == moe.MOE_EINVAL
