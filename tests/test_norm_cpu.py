"""Refusals of the RMS norm: every argument error is found on the host, before
anything is enqueued (no GPU needed)."""
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
    base = dict(R=4, K=256, dtype=0, weight_dtype=0, fmt=0, group=128, eps=1e-6)
    base.update(kw)
    return C.byref(moe.MoeNormCfg(*[base[n] for n, _ in moe.MoeNormCfg._fields_]))


def norm(c, x=FAKE, r=FAKE, w=FAKE, y=FAKE, s=FAKE, rstd=FAKE):
    return moe.raw_call("moe_rms_norm", c, x, r, w, y, s, rstd, None)


def quant(c, x=FAKE, r=FAKE, w=FAKE, y=FAKE, s=FAKE, q=FAKE, qs=FAKE):
    return moe.raw_call("moe_rms_norm_quant", c, x, r, w, y, s, q, qs, None)


def grad(c, dy=FAKE, ds=FAKE, s=FAKE, rstd=FAKE, w=FAKE, dx=FAKE, dw=FAKE, work=FAKE, nb=1 << 30):
    return moe.raw_call("moe_rms_norm_backward", c, dy, ds, s, rstd, w, dx, dw, work, nb, None)


CALLS = {"norm": norm, "quant": quant, "grad": grad}


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(name):
    call = CALLS[name]
    assert call(None) == moe.MOE_ERR_NULL_ARG
    required = {"norm": ("x", "w", "y"), "quant": ("x", "w", "q", "qs"), "grad": ("dy", "s", "rstd", "w", "work")}[name]
    for n in required:
        assert call(cfg(), **{n: None}) == moe.MOE_ERR_NULL_ARG, n
        assert call(cfg(K=7), **{n: None}) == moe.MOE_ERR_NULL_ARG, n  # NULL comes before the shape
    for kw in (dict(R=-1), dict(R=(1 << 31) - 1023), dict(K=0), dict(K=4), dict(K=260), dict(K=(1 << 14) + 8)):
        assert call(cfg(**kw)) == moe.MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(dtype=2), dict(dtype=-1), dict(weight_dtype=1), dict(weight_dtype=3), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=2.0)):
        assert call(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw
    names = {"norm": "x r w y s rstd", "quant": "x r w y s q qs", "grad": "dy ds s rstd w dx dw work"}[name]
    for n in names.split():
        assert call(cfg(), **{n: FAKE + 8}) == moe.MOE_ERR_MISALIGNED, n


def test_quant_formats():
    for kw in (dict(fmt=3), dict(fmt=-1), dict(group=64), dict(group=0), dict(group=256)):
        assert quant(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(K=288), dict(K=264, group=32), dict(K=264, fmt=1), dict(K=272, fmt=2)):
        assert quant(cfg(**kw)) == moe.MOE_ERR_BAD_SHAPE, kw


def test_no_rows():
    assert norm(cfg(R=0), x=None, r=None, y=None, s=None, rstd=None) == moe.MOE_OK
    assert quant(cfg(R=0), x=None, r=None, y=None, s=None, q=None, qs=None) == moe.MOE_OK
    assert grad(cfg(R=0), dy=None, ds=None, s=None, rstd=None, dx=None, dw=None, work=None, nb=0) == moe.MOE_OK


def test_workspace():
    n = C.c_size_t(0)
    size = lambda c: moe.raw_call("moe_rms_norm_backward_workspace_size", c, C.byref(n))
    assert size(cfg(R=4, K=4096)) == moe.MOE_OK and n.value == 4 * 4096 * 4
    assert size(cfg(R=0)) == moe.MOE_OK and n.value == 0
    assert size(None) == moe.MOE_ERR_NULL_ARG and size(cfg(K=4)) == moe.MOE_ERR_BAD_SHAPE
    assert size(cfg(dtype=2)) == moe.MOE_ERR_UNSUPPORTED
    assert moe.raw_call("moe_rms_norm_backward_workspace_size", cfg(), None) == moe.MOE_ERR_NULL_ARG
    assert grad(cfg(K=4096), nb=4 * 4096 * 4 - 1) == moe.MOE_ERR_WORKSPACE
    assert size(cfg(R=1 << 20, K=1 << 14)) == moe.MOE_OK and n.value < 1 << 26  # does not grow with the rows


def test_python_refusals():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for f in (moe.moe_rms_norm, moe.moe_rms_norm_quant):
        with pytest.raises(ValueError, match="GPU"):
            f(x, w)
        for bad in ((x[0], w), (x.float(), w.float()), (x, w.half()), (x, w[:32]), (x, w, x[:2]), (x, w, x.half())):
            with pytest.raises(ValueError):
                f(*bad)
        with pytest.raises(ValueError, match="needs a residual"):
            f(x, w, sum_out=x)
    with pytest.raises(ValueError, match="no gradient"):
        moe.moe_rms_norm_quant(x, w.clone().requires_grad_())
    with pytest.raises(ValueError, match="where a gradient is needed"):
        moe.moe_rms_norm(x.clone().requires_grad_(), w, out=x)
    with pytest.raises(ValueError, match="no gradient"):
        moe.moe_rms_norm_backward(x.clone().requires_grad_(), None, x, torch.ones(4), w)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="forward-mode"):
            moe.moe_rms_norm(dual, w)
        with pytest.raises(ValueError, match="forward-mode"):
            moe.moe_rms_norm_quant(x, w, dual)
