"""A workspace for T tokens serves a batch of fewer tokens of the same dims, in the few-token layer too (no GPU)."""
import pytest

# the last three: the few-token layer's rows of h outweigh moe_forward's whole workspace
DIMS = [(2688, 128, 6, 1856), (256, 8, 2, 128), (64, 16, 16, 16), (64, 256, 16, 4096), (16, 4, 4, 65536), (32, 64, 8, 1024)]


@pytest.mark.parametrize("kw", [{}, dict(fp8=True), dict(fp8_b128=True), dict(nvfp4=True), dict(shared=True)], ids=str)
@pytest.mark.parametrize("H,E,K,F", DIMS)
def test_never_smaller_for_more_tokens(H, E, K, F, kw):
    import routed_expert_moe_b200 as moe
    kw = dict(kw)
    if kw.pop("shared", False):
        kw["Fs"], K, E = F, min(K, 15), min(E, 255)
    if kw.get("nvfp4") and (H % 32 or F % 32):
        pytest.skip("NVFP4 rows are multiples of 32")
    sizes = [moe.workspace_size(moe.dims(T, H, E, K, F, **kw)) for T in [*range(1, 80), 96, 128, 300, 577, 1024, 4096]]
    assert sizes == sorted(sizes)
