"""Refusals of the row-major products at the size of a launch, found on the host
before anything is enqueued (no GPU needed)."""
import pytest

import bit_grouped_gemm_amd as moe
from test_mm_cpu import FAKE, cfg, lib  # noqa: F401 (the fixture builds and loads the library)


@pytest.mark.parametrize("kw", [dict(R=(1 << 31) - 1024, N=512, K=512, E=1), dict(R=1 << 30, N=1024, K=1024, E=1),
                                dict(R=1 << 24, N=1 << 16, K=1 << 16, E=7)], ids=str)
def test_more_tiles_than_a_launch_has(kw):
    """2^24 tiles of 256 x 256: fewer than 2^31 workgroups, but of 512 threads each, 2^33 work items."""
    for name in ("moe_grouped_mm", "moe_grouped_mm_dgrad"):
        assert moe.raw_call(name, cfg(**kw), FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_BAD_SHAPE, name
    assert moe.raw_call("moe_mm_i8", cfg(**kw), FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                        None) == moe.MOE_ERR_BAD_SHAPE
    assert moe.raw_call("moe_linear_i8", cfg(**kw), FAKE, 0, FAKE, FAKE, FAKE, None, FAKE, FAKE, 1 << 62,
                        None) == moe.MOE_ERR_BAD_SHAPE
