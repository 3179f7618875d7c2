"""The structs of scales hold device pointers: the tensors that they were made of live as long as they do (no GPU)."""
import gc
import weakref

import pytest
import torch


@pytest.mark.parametrize("make,n", [("fp8_scales", 2), ("nvfp4_scales", 4)])
def test_scales_live_as_long_as_their_struct(make, n):
    import routed_expert_moe_b200 as moe
    t = [torch.ones(8) for _ in range(n)]
    alive = [weakref.ref(v) for v in t]
    first = t[0].data_ptr()
    sc = getattr(moe, make)(*t[:2], 1.0, 1.0, *t[2:])
    del t
    gc.collect()
    assert all(a() is not None for a in alive) and sc.w_up_scale == first
    del sc
    gc.collect()
    assert all(a() is None for a in alive)
