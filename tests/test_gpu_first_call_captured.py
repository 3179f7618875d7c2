"""The library's first call in a process is one that a graph captures: nothing of its set-up may end the capture."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]

SCRIPT = """
import sys
import torch
import routed_expert_moe_b200 as moe
bf = torch.bfloat16
torch.manual_seed(1)
r = lambda *s: torch.randn(*s, device="cuda").to(bf)
T, H, E, K, F = 3, 256, 8, 2, 128
d = moe.dims(T, H, E, K, F)
x, wr, wu, wd, gain = r(T, H), r(E, H), r(E, F, H), r(E, H, F), r(H)
ws = moe.alloc_workspace(d)
codes = torch.randint(0, 120, (200, H), device="cuda", dtype=torch.uint8)
scales = torch.ones(200, H // 128, device="cuda")
out = {"few": torch.empty(T, H, device="cuda", dtype=bf), "norm": torch.empty(T, H, device="cuda", dtype=bf),
       "linear": torch.empty(5, 200 // 16 * 16, device="cuda", dtype=bf),
       "tiles": torch.empty(40, 200 // 16 * 16, device="cuda", dtype=bf)}
n = out["linear"].shape[1]
calls = {"few": lambda: moe.forward_few(d, x, wr, None, wu, wd, out["few"], ws),
         "norm": lambda: moe.prenorm(x, gain, u=out["norm"]),
         "linear": lambda: moe.linear_fp8_b128(codes[:5], scales[:5], codes[:n], scales[:n], out["linear"]),
         "tiles": lambda: moe.linear_fp8_b128(codes[:40], scales[:40], codes[:n], scales[:n], out["tiles"])}
order = sys.argv[1:]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for k in order:
        calls[k]()
graph.replay()
torch.cuda.synchronize()
got = {k: out[k].clone() for k in order}
for k in order:
    out[k].zero_()
    calls[k]()
torch.cuda.synchronize()
moe.check_device_error()
assert all(torch.equal(out[k], got[k]) and float(got[k].abs().max()) > 0 for k in order)
del graph
"""


@pytest.mark.parametrize("order", [["few"], ["norm"], ["linear"], ["tiles"], ["norm", "linear", "tiles", "few"]], ids="-".join)
def test_first_call_is_captured(order):
    run = subprocess.run([sys.executable, "-c", SCRIPT, *order], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]
