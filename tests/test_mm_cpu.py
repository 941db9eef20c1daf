"""Refusals of the row-major products and the int8 quantiser: every argument
error is found on the host, before anything is enqueued (no GPU needed)."""
import ctypes as C
import os

import pytest
import torch

import bit_grouped_gemm_amd as moe

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its host checks first


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from bit_grouped_gemm_amd import build
        build.build()
    return moe.load()


def cfg(**kw):
    base = dict(R=4, N=64, K=64, E=2, T=4, dtype=0, out_dtype=0, clear_rest=0)
    base.update(kw)
    return C.byref(moe.MoeMmCfg(*[base[n] for n, _ in moe.MoeMmCfg._fields_]))


GROUPED = ("moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad")


@pytest.mark.parametrize("name", GROUPED)
def test_grouped_refusals(name):
    work = (None, 0) if name == "moe_grouped_mm_wgrad" else ()
    call = lambda c, p=FAKE, q=FAKE, o=FAKE, out=FAKE: moe.raw_call(name, c, p, q, o, out, *work, None)
    assert call(None) == moe.MOE_ERR_NULL_ARG
    for kw in (dict(p=None), dict(q=None), dict(o=None), dict(out=None)):
        assert call(cfg(), **kw) == moe.MOE_ERR_NULL_ARG, kw
    # NULL comes before the shape
    assert call(cfg(N=7), p=None) == moe.MOE_ERR_NULL_ARG
    for kw in (dict(R=-1), dict(R=(1 << 31) - 1023), dict(N=0), dict(K=0), dict(E=0), dict(E=1025), dict(N=60), dict(K=12), dict(N=(1 << 20) + 8),
               dict(K=(1 << 20) + 8), dict(clear_rest=2)):
        assert call(cfg(**kw)) == moe.MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(dtype=2, out_dtype=2), dict(dtype=3), dict(out_dtype=1), dict(dtype=1, out_dtype=0),
               dict(out_dtype=-1)):
        assert call(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(p=FAKE + 8), dict(q=FAKE + 2), dict(o=FAKE + 2), dict(out=FAKE + 8)):
        assert call(cfg(), **kw) == moe.MOE_ERR_MISALIGNED, kw


def test_grouped_refuses_more_workgroups_than_a_launch_has():
    # 2^31 - 1024 rows of 2^20 outputs: the tile count passes 2^31
    assert moe.raw_call("moe_grouped_mm", cfg(R=(1 << 31) - 1024, N=1 << 20, E=1), FAKE, FAKE, FAKE, FAKE,
                        None) == moe.MOE_ERR_BAD_SHAPE


def test_wgrad_workspace():
    """Few small matrices split their rows and need scratch; many tiles or few rows need none."""
    n = C.c_size_t(0)
    size = lambda c: moe.raw_call("moe_grouped_mm_wgrad_workspace_size", c, C.byref(n))
    assert size(cfg(R=1 << 15, N=512, K=512, E=1)) == moe.MOE_OK and n.value == 64 * 512 * 512 * 4
    need = n.value
    for kw in (dict(R=1 << 15, N=4096, K=4096, E=1), dict(R=512, N=512, K=512, E=1), dict(R=0, E=1)):
        assert size(cfg(**kw)) == moe.MOE_OK and n.value == 0, kw
    assert size(None) == moe.MOE_ERR_NULL_ARG
    assert moe.raw_call("moe_grouped_mm_wgrad_workspace_size", cfg(), None) == moe.MOE_ERR_NULL_ARG
    assert size(cfg(N=4)) == moe.MOE_ERR_BAD_SHAPE and size(cfg(dtype=2, out_dtype=2)) == moe.MOE_ERR_UNSUPPORTED
    call = lambda work, nb: moe.raw_call("moe_grouped_mm_wgrad", cfg(R=1 << 15, N=512, K=512, E=1), FAKE, FAKE, FAKE,
                                         FAKE, work, nb, None)
    assert call(None, need) == moe.MOE_ERR_NULL_ARG
    assert call(FAKE, need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(FAKE + 8, need) == moe.MOE_ERR_MISALIGNED


def test_quant_refusals():
    call = lambda R=4, K=64, dt=0, glu=0, x=FAKE, q=FAKE, s=FAKE: moe.raw_call("moe_quant_i8", R, K, dt, glu, x, q, s,
                                                                             None)
    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert call(**kw) == moe.MOE_ERR_NULL_ARG, kw
    for kw in (dict(R=-1), dict(K=0), dict(K=8), dict(K=(1 << 20) + 16)):
        assert call(**kw) == moe.MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(dt=2), dict(dt=-1), dict(glu=2)):
        assert call(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(x=FAKE + 2), dict(q=FAKE + 8), dict(s=FAKE + 4)):
        assert call(**kw) == moe.MOE_ERR_MISALIGNED, kw
    assert call(R=0, x=None, q=None, s=None) == moe.MOE_OK


def test_mm_i8_refusals():
    call = lambda c, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, o=FAKE, t=None, y=FAKE: moe.raw_call(
        "moe_mm_i8", c, xq, xs, wq, ws, o, t, y, None)
    assert call(None) == moe.MOE_ERR_NULL_ARG
    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y=None)):
        assert call(cfg(), **kw) == moe.MOE_ERR_NULL_ARG, kw
    for kw in (dict(K=72), dict(K=(1 << 16) + 16), dict(N=60), dict(R=-1), dict(E=0)):
        assert call(cfg(**kw)) == moe.MOE_ERR_BAD_SHAPE, kw
    assert call(cfg(), o=None) == moe.MOE_ERR_BAD_SHAPE               # two groups need offsets
    assert call(cfg(T=-1), t=FAKE) == moe.MOE_ERR_BAD_SHAPE
    assert call(cfg(T=1 << 25), t=FAKE) == moe.MOE_ERR_BAD_SHAPE      # T * K reaches 2^31
    for kw in (dict(out_dtype=3), dict(out_dtype=-1)):
        assert call(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(xq=FAKE + 8), dict(xs=FAKE + 4), dict(wq=FAKE + 8), dict(ws=FAKE + 4), dict(o=FAKE + 2),
               dict(t=FAKE + 1), dict(y=FAKE + 8)):
        assert call(cfg(), **kw) == moe.MOE_ERR_MISALIGNED, kw


def test_linear_i8_refusals():
    n = C.c_size_t(0)
    size = lambda c, g=0: moe.raw_call("moe_linear_i8_workspace_size", c, g, C.byref(n))
    assert size(cfg(R=5, K=48)) == moe.MOE_OK and n.value == 256 + 256
    assert size(cfg(R=5, K=48, T=100), 1) == moe.MOE_OK and n.value == 4864 + 512
    for kw in (dict(R=0), dict(R=1, K=8192), dict(R=1, K=8192, T=50)):  # one row: no codes outside the kernel
        assert size(cfg(**kw), int("T" in kw)) == moe.MOE_OK and n.value == 0, kw
    assert size(cfg(R=1, K=8208)) == moe.MOE_OK and n.value == 8448 + 256
    assert size(None) == moe.MOE_ERR_NULL_ARG
    assert moe.raw_call("moe_linear_i8_workspace_size", cfg(), 0, None) == moe.MOE_ERR_NULL_ARG
    for c, g in ((cfg(K=24), 0), (cfg(T=-1), 1), (cfg(), 2)):
        assert size(c, g) == moe.MOE_ERR_BAD_SHAPE
    call = lambda c, x=FAKE, glu=0, wq=FAKE, ws=FAKE, o=FAKE, t=None, y=FAKE, work=FAKE, nb=1 << 20: moe.raw_call(
        "moe_linear_i8", c, x, glu, wq, ws, o, t, y, work, nb, None)
    assert call(None) == moe.MOE_ERR_NULL_ARG
    for kw in (dict(x=None), dict(wq=None), dict(ws=None), dict(y=None), dict(work=None)):
        assert call(cfg(R=5), **kw) == moe.MOE_ERR_NULL_ARG, kw
    assert call(cfg(K=24)) == moe.MOE_ERR_BAD_SHAPE
    assert call(cfg(), o=None) == moe.MOE_ERR_BAD_SHAPE
    for kw in (dict(dtype=2), dict(out_dtype=4)):
        assert call(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw
    assert call(cfg(), glu=2) == moe.MOE_ERR_UNSUPPORTED
    assert call(cfg(), work=FAKE + 8) == moe.MOE_ERR_MISALIGNED
    assert call(cfg(R=5), nb=767) == moe.MOE_ERR_WORKSPACE  # 512 + 256


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_python_refusals():
    """Types, shapes and devices are checked before any pointer is taken."""
    off = t(3, dtype=torch.int32)
    x, w, dy = t(4, 64), t(2, 32, 64), t(4, 32)
    bad = [
        lambda: moe.moe_grouped_mm(x.float(), w.float(), off),
        lambda: moe.moe_grouped_mm(x, w.half(), off),
        lambda: moe.moe_grouped_mm(x, t(2, 32, 72), off),
        lambda: moe.moe_grouped_mm(x, w[0], off),
        lambda: moe.moe_grouped_mm(x, w, off.long()),
        lambda: moe.moe_grouped_mm(x, w, off[:2]),
        lambda: moe.moe_grouped_mm(x, w, off, out=t(4, 40)),
        lambda: moe.moe_grouped_mm(x, w, off, out=t(4, 32, dtype=torch.float16)),
        lambda: moe.moe_grouped_mm(x.clone().requires_grad_(), w, off, out=t(4, 32)),
        lambda: moe.moe_grouped_mm(x.clone().requires_grad_(), w, off, out_dtype=torch.float32),
        lambda: moe.moe_grouped_mm_dgrad(dy, t(2, 40, 64), off),
        lambda: moe.moe_grouped_mm_wgrad(dy, t(5, 64), off),
        lambda: moe.moe_grouped_mm_wgrad(dy, x, off[:1]),
        lambda: moe.moe_quant_i8(x.float()),
        lambda: moe.moe_quant_i8(t(4, 63), swiglu=True),
        lambda: moe.moe_quant_i8(x, codes=t(4, 32, dtype=torch.int8)),
        lambda: moe.moe_mm_i8(x, t(4, dtype=torch.float32), w.to(torch.int8), t(2, 32, dtype=torch.float32), off),
        lambda: moe.moe_mm_i8(x.to(torch.int8), t(5, dtype=torch.float32), w.to(torch.int8),
                              t(2, 32, dtype=torch.float32), off),
        lambda: moe.moe_mm_i8(x.to(torch.int8), t(4, dtype=torch.float32), w.to(torch.int8),
                              t(2, 32, dtype=torch.float32)),                       # three dimensions need offsets
        lambda: moe.moe_mm_i8(x.to(torch.int8), t(4, dtype=torch.float32), w[0].to(torch.int8),
                              t(32, dtype=torch.float32), out_dtype=torch.float64),
        lambda: moe.moe_linear_i8(x, w[0, :, :48].contiguous().to(torch.int8), t(32, dtype=torch.float32)),
        lambda: moe.moe_linear_i8(x, w[0].to(torch.int8), t(32, dtype=torch.float32), swiglu=True),
        lambda: moe.moe_grouped_mm(t(1, 8).expand(1 << 31, 8), w, off),             # more rows than an int32 counts
        lambda: moe.moe_quant_i8(t(1, 16).expand(1 << 32, 16)),
        # tensors that are no GPU's are refused, not computed elsewhere
        lambda: moe.moe_grouped_mm(x, w, off),
        lambda: moe.moe_quant_i8(x),
    ]
    for i, f in enumerate(bad):
        try:
            f()
        except ValueError:
            continue
        raise AssertionError(f"call {i} was not refused")
