"""The exact layers themselves (no GPU): sums that fp32 holds, and outputs that a lost rounding or value changes."""
import pytest

import _exact_layer as X


@pytest.mark.parametrize("fmt,T,H,E,K,F,ns", X.cases())
def test_sums_fit_and_planted_mistakes_show(fmt, T, H, E, K, F, ns):
    s = X.make(T, H, E, K, F, fmt, ns, seed=T + H)
    out, big = X.output(s)
    assert big < 2 ** 24
    want = out.bfloat16()
    assert float((want != 0).double().mean()) > 0.2
    plants = ["y8", "up_tail", "down_tail"] + (["h8"] if fmt == "bf16" else [])
    for plant in plants:
        wrong = (X.output(s, plant)[0].bfloat16() != want).double().mean()
        assert float(wrong) > 0.05, (plant, float(wrong))
