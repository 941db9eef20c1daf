"""Argument checks of the MFMA-rate probe's 32x32x64 form (no GPU needed)."""
import ctypes as C

import bit_grouped_gemm_amd as moe

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its host checks first


def test_argument_errors():
    moe.load()
    fl = C.c_double(0.0)
    call = lambda wfmt, iters, sink, sn: moe.raw_call("moe_mfma_rate", wfmt, iters, sink, C.c_size_t(sn), C.byref(fl), None)
    form = moe.RATE_E2M1_E2M1_32
    assert call(form, 16, None, 1 << 12) == moe.MOE_ERR_NULL_ARG
    assert call(form, 16, FAKE + 4, 1 << 12) == moe.MOE_ERR_MISALIGNED
    assert call(form + 1, 16, FAKE, 1 << 12) == moe.MOE_ERR_UNSUPPORTED
    assert call(form, 0, FAKE, 1 << 12) == moe.MOE_ERR_BAD_SHAPE
    assert call(form, 65537, FAKE, 1 << 12) == moe.MOE_ERR_BAD_SHAPE
    assert call(form, 16, FAKE, 16) == moe.MOE_ERR_WORKSPACE
