"""Loads of the kernels (no GPU).  They start while the preceding one still runs (programmatic dependent launch), so
what that one writes - codes and scales of a norm or a quantiser, a permutation, weights quantised just before -
changes while they exist.  A read-only load may not be used on such memory, and a restrict pointer to const lets
the compiler choose one."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "routed_expert_moe_b200" / "csrc"
READ_ONLY = re.compile(r"\b__ldg\s*\(|ld\.global(\.\w+)*\.nc\b|\bconst\b[^;,(]*\*\s*__restrict__")


@pytest.mark.parametrize("name", sorted(p.name for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh", ".h")))
def test_no_read_only_loads(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    assert READ_ONLY.findall(text) == []
