"""Loads of the few-token layer and the FP8_B128 product (no GPU).  Their kernels start while the preceding one
still runs (programmatic dependent launch), so what that one writes - codes and scales of a norm or a quantiser,
weights quantised just before - changes while they exist.  A read-only load may not be used on such memory."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "routed_expert_moe_b200" / "csrc"
READ_ONLY = re.compile(r"\b__ldg\s*\(|ld\.global(\.\w+)*\.nc\b|\bconst\b[^;,(]*\*\s*__restrict__")


@pytest.mark.parametrize("name", ["few.cu", "linear_b128.cu", "weight_stream.cuh", "norm.cu", "common.cuh"])
def test_no_read_only_loads(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert READ_ONLY.findall(text) == []
