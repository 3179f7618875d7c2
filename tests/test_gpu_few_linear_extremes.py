"""The few-token layer and the FP8_B128 product at the ends of their documented ranges, against the float64 forms."""
import pytest
import torch

from test_gpu_few import Layer
from test_gpu_linear_b128 import check, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "b128"])
@pytest.mark.parametrize("T,H,E,K,F", [(16, 65536, 2, 1, 16), (3, 65536, 2, 2, 32), (16, 16, 2, 1, 65536), (1, 16, 1, 1, 65536),
                                       (1, 16, 1, 1, 16), (16, 16, 256, 16, 16), (16, 32, 256, 1, 272)])
def test_layer(moe, T, H, E, K, F, fmt):
    Layer(moe, T, H, E, K, F, fmt, residual=True, seed=T + H + F, std=0.02).check()


@pytest.mark.parametrize("M,N,K", [(1, 1 << 20, 16), (16, 1 << 20, 16), (17, 1 << 20, 16), (1, 16, 65536), (16, 32, 65536),
                                   (17, 16, 65536), (130, 32, 65536), (1, 16, 16), (40000, 16, 16)])
def test_product(moe, M, N, K):
    xq, xs, wq, ws = operands(M, N, K, M + N + K)
    out = torch.full((M, N), 3.0, device="cuda", dtype=torch.bfloat16)
    moe.linear_fp8_b128(xq, xs, wq, ws, out)
    moe.check_device_error()
    check(out, xq, xs, wq, ws, None)
