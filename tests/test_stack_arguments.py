"""Refusals of the stack's options, before anything reaches a GPU."""
import pytest

pytest.importorskip("torch")


def bare(T, **kw):
    from routed_expert_moe_b200.stack import MoeStack
    return MoeStack(T, 64, 4, 2, 32, device="cpu", **kw)


def test_few_has_a_limit():
    with pytest.raises(ValueError, match="at most"):
        bare(17, few=True)


@pytest.mark.parametrize("kw", [{"gate": 1}, {"gain_pre": 1}, {"alpha": 0.5}, {"shared": (1, 2)}])
def test_parts_of_a_sandwich_need_its_gain(kw):
    with pytest.raises(ValueError, match="gain_post"):
        bare(4, fp8=False).add_layer(None, None, None, **kw)


def test_few_takes_the_shapes_of_its_dims(monkeypatch):
    """Wrong types, shapes and strides of the few-token layer's tensors."""
    import torch
    import routed_expert_moe_b200 as moe
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # CPU tensors stand for the current device's
    bf = torch.bfloat16
    T, H, E, K, F = 3, 64, 8, 2, 48
    d = moe.dims(T, H, E, K, F)
    ok = dict(x=torch.zeros(T, H, dtype=bf), w_router=torch.zeros(E, H, dtype=bf), bias=torch.zeros(E),
              w_up=torch.zeros(E, F, H, dtype=bf), w_down=torch.zeros(E, H, F, dtype=bf),
              out=torch.zeros(T, H, dtype=bf), ws=torch.zeros(256, dtype=torch.uint8), topk_idx=None)
    bad = [dict(x=torch.zeros(T + 1, H, dtype=bf)), dict(x=torch.zeros(T, H)), dict(w_router=torch.zeros(H, E, dtype=bf)),
           dict(bias=torch.zeros(E, dtype=bf)), dict(w_up=torch.zeros(E, H, F, dtype=bf)),
           dict(w_down=torch.zeros(E, F, H, dtype=bf).transpose(1, 2)), dict(out=torch.zeros(T, 2 * H, dtype=bf)[:, ::2]),
           dict(topk_idx=torch.zeros(T, K, dtype=torch.int64))]
    for change in bad:
        with pytest.raises(moe.MoeError, match="moe_forward_few: needs"):
            moe.forward_few(d, **{**ok, **change})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)    # another device than the tensors'
    with pytest.raises(moe.MoeError, match="moe_forward_few: needs"):
        moe.forward_few(d, **ok)
