"""Types, shapes, strides and devices of the norms' and the FP8_B128 product's tensors, checked before the call: every
argument is right but the one under test (no GPU)."""
import re

import pytest
import torch

BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32
T, H, KP = 3, 272, 384


@pytest.fixture
def moe(monkeypatch):
    import routed_expert_moe_b200 as m
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # CPU tensors stand for the current device's
    return m


def rows(dtype=BF, t=T, h=H):
    return torch.zeros(t, h, dtype=dtype)


PRE = dict(x=rows, gain=lambda: torch.zeros(H, dtype=BF), u=rows, codes=lambda: rows(U8, h=KP),
           scales=lambda: rows(F32, h=KP // 128))
POST = dict(PRE, y=rows, gate=rows, x_out=rows, next_gain=lambda: torch.zeros(H, dtype=BF))
LIN = dict(x_codes=lambda: rows(U8, 5, 256), x_scales=lambda: rows(F32, 5, 2), w_codes=lambda: rows(U8, 64, 256),
           w_scales=lambda: rows(F32, 64, 2), out=lambda: rows(BF, 5, 64))


def wrong(make, first):
    """The same tensor with a wrong type, with a row or a column more, and with strides."""
    t = make()
    out = [t.to(torch.float16), torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]]
    if not first:                            # the first argument's shape is what the others are measured by
        out.append(torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype))
        if t.dim() == 2:
            out.append(torch.zeros(t.shape[0] + 1, t.shape[1], dtype=t.dtype))
    return out


def cases():
    for call, args, first in (("prenorm", PRE, ("x",)), ("postnorm", POST, ("x",)),
                              ("linear_fp8_b128", LIN, ("x_codes", "w_codes"))):
        for name in args:
            for i in range(len(wrong(args[name], name in first))):
                yield pytest.param(call, args, name, i, name in first, id=f"{call}-{name}-{i}")


@pytest.mark.parametrize("call,args,name,i,first", list(cases()))
def test_one_wrong_argument(moe, call, args, name, i, first):
    good = {k: make() for k, make in args.items()}
    bad = dict(good, **{name: wrong(args[name], first)[i]})
    with pytest.raises(moe.MoeError, match=f"moe_{call}: needs a contiguous"):
        getattr(moe, call)(**bad)


@pytest.mark.parametrize("call,args", [("prenorm", PRE), ("postnorm", POST), ("linear_fp8_b128", LIN)])
def test_another_device(moe, monkeypatch, call, args):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(moe.MoeError, match=f"moe_{call}: needs a contiguous"):
        getattr(moe, call)(**{k: make() for k, make in args.items()})


@pytest.mark.parametrize("change,text", [(dict(act="gelu"), "act 'gelu'"), (dict(act=1), "act 1"),
                                         (dict(x_codes=rows(U8, 5, 200)), "code rows of 200")])
def test_product_options(moe, change, text):
    with pytest.raises(moe.MoeError, match=re.escape(text)):
        moe.linear_fp8_b128(**dict({k: make() for k, make in LIN.items()}, **change))
