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
