"""Scales at an address that no fp32 value may have: refused on the host, in every format and call that takes them (no
GPU; every call here is one that has to be refused)."""
import ctypes

import pytest

FAR = [ctypes.c_void_p(i << 32) for i in range(1, 9)]


@pytest.mark.parametrize("call", ["moe_forward", "moe_forward_few", "moe_expert_ffn"])
@pytest.mark.parametrize("kw", [dict(fp8=True), dict(fp8_b128=True), dict(nvfp4=True)], ids=str)
@pytest.mark.parametrize("which", ["w_up_scale", "w_down_scale"])
def test_refused(call, kw, which):
    import routed_expert_moe_b200 as moe
    if call == "moe_forward_few" and "nvfp4" in kw:
        pytest.skip("not a format of the few-token layer")
    d = moe.dims(4, 2688, 128, 6, 1856, **kw)
    sc = moe.MoeFp8Scales(1 << 20, 2 << 20, 1.0, 1.0, 3 << 20, 4 << 20)
    setattr(sc, which, getattr(sc, which) + 2)
    x, wr, wu, wd, out, ws, a, b = FAR
    lib, n = moe.raw_library(), 1 << 30
    if call == "moe_expert_ffn":
        got = lib.moe_expert_ffn(ctypes.byref(d), x, a, b, wu, wd, None, None, ctypes.byref(sc), out, ws, n, None)
    else:
        got = getattr(lib, call)(ctypes.byref(d), x, wr, None, wu, wd, None, None, ctypes.byref(sc), None, out, None, None,
                                 ws, n, None)
    assert got == moe.MOE_EINVAL
