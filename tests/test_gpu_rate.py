"""The MFMA-rate probe's 32x32x64 form computes what it claims (needs an MI355X)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("iters", [1, 777, 65536])
def test_mfma_rate_of_the_32_form(iters):
    """Every workgroup's sum is exactly 4096 * iters, and the FLOP count matches the grid."""
    import bit_grouped_gemm_amd as moe
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sink = torch.full((8192,), -1.0, device="cuda")
    flops = moe.moe_mfma_rate(moe.RATE_E2M1_E2M1_32, iters, sink)
    torch.cuda.synchronize()
    grid = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    assert flops == grid * 4 * iters * 4 * (32 * 32 * 64 * 2)
    assert (sink[:grid] == 4096.0 * iters).all() and (sink[grid:] == -1.0).all()
