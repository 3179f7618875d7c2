"""The few-token layer's scales and workspace: type, size and device, checked before the call like its other tensors (no
GPU; every argument is right but the one under test)."""
import pytest
import torch

T, H, E, K, F = 3, 272, 8, 2, 144
BF, U8 = torch.bfloat16, torch.uint8


def layer(moe, fmt):
    b128 = fmt == "b128"
    kh, kf = (384, 256) if b128 else (H, F)
    d = moe.dims(T, H, E, K, F, fp8=not b128, fp8_b128=b128)
    su, sd = (torch.ones(E, F, 3), torch.ones(E, H, 2)) if b128 else (torch.ones(E), torch.ones(E))
    return d, dict(x=torch.zeros(T, H, dtype=BF), w_router=torch.zeros(E, H, dtype=BF), bias=None,
                   w_up=torch.zeros(E, F, kh, dtype=U8), w_down=torch.zeros(E, H, kf, dtype=U8),
                   out=torch.zeros(T, H, dtype=BF), ws=torch.zeros(1 << 20, dtype=U8)), su, sd


@pytest.fixture
def moe(monkeypatch):
    import routed_expert_moe_b200 as m
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # CPU tensors stand for the current device's
    return m


@pytest.mark.parametrize("fmt", ["e4m3", "b128"])
def test_scales(moe, fmt):
    d, a, su, sd = layer(moe, fmt)
    bad = [(su.double(), sd), (su, sd.half()), (su[:-1], sd), (su, torch.cat([sd, sd])), (sd if fmt == "b128" else su[:1], sd),
           (torch.stack([su, su], -1)[..., 0], sd)]
    for s in bad:
        with pytest.raises(moe.MoeError, match="moe_forward_few: needs"):
            moe.forward_few(d, **a, scales=moe.fp8_scales(*s, 1.0, 1.0))


def test_workspace(moe):
    d, a, su, sd = layer(moe, "e4m3")
    sc = moe.fp8_scales(su, sd, 1.0, 1.0)
    class Elsewhere:   # a workspace of another device
        device = "cuda:5"

        def get_device(self):
            return 5

        def is_contiguous(self):
            return True

    for ws in (Elsewhere(), torch.zeros(1 << 20, dtype=U8)[::2]):
        with pytest.raises(moe.MoeError, match="workspace"):
            moe.forward_few(d, **{**a, "ws": ws}, scales=sc)
