"""Refusals of the row-major MXFP4 operators: every argument error is found on
the host, before anything is enqueued (no GPU needed)."""
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


def quant(R=4, K=64, dt=0, glu=0, x=FAKE, q=FAKE, s=FAKE):
    return moe.raw_call("moe_quant_mx4", R, K, dt, glu, x, q, s, None)


def mm(c, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, o=FAKE, t=None, y=FAKE):
    return moe.raw_call("moe_mm_mx4", c, xq, xs, wq, ws, o, t, y, None)


def linear(c, x=FAKE, glu=0, wq=FAKE, ws=FAKE, o=FAKE, t=None, y=FAKE, work=FAKE, nb=1 << 50):
    return moe.raw_call("moe_linear_mx4", c, x, glu, wq, ws, o, t, y, work, nb, None)


def test_quant_refusals():
    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert quant(**kw) == moe.MOE_ERR_NULL_ARG and quant(K=7, **kw) == moe.MOE_ERR_NULL_ARG, kw
    for kw in (dict(R=-1), dict(K=0), dict(K=16), dict(K=48), dict(K=(1 << 20) + 32)):
        assert quant(**kw) == moe.MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(dt=2), dict(dt=-1), dict(glu=2)):
        assert quant(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(x=FAKE + 2), dict(q=FAKE + 8), dict(s=FAKE + 4)):
        assert quant(**kw) == moe.MOE_ERR_MISALIGNED, kw
    assert quant(R=0, x=None, q=None, s=None) == moe.MOE_OK


@pytest.mark.parametrize("call,tensors", [(mm, ("xq", "xs", "wq", "ws", "y")), (linear, ("x", "wq", "ws", "y", "work"))],
                         ids=["mm", "linear"])
def test_product_refusals(call, tensors):
    assert call(None) == moe.MOE_ERR_NULL_ARG
    for n in tensors:
        assert call(cfg(), **{n: None}) == moe.MOE_ERR_NULL_ARG, n
        assert call(cfg(K=7), **{n: None}) == moe.MOE_ERR_NULL_ARG, n  # NULL comes before the shape
        assert call(cfg(), **{n: FAKE + 8}) == moe.MOE_ERR_MISALIGNED, n
    assert call(cfg(), o=FAKE + 2) == moe.MOE_ERR_MISALIGNED and call(cfg(), t=FAKE + 1) == moe.MOE_ERR_MISALIGNED
    for kw in (dict(R=-1), dict(R=(1 << 31) - 1023), dict(N=0), dict(N=60), dict(K=0), dict(K=48), dict(E=0),
               dict(E=1025), dict(N=(1 << 20) + 8), dict(K=(1 << 20) + 32), dict(clear_rest=2),
               dict(R=(1 << 31) - 1024, N=1 << 20, E=1)):
        assert call(cfg(**kw)) == moe.MOE_ERR_BAD_SHAPE, kw
    assert call(cfg(), o=None) == moe.MOE_ERR_BAD_SHAPE              # two groups need offsets
    assert call(cfg(T=-1), t=FAKE) == moe.MOE_ERR_BAD_SHAPE
    assert call(cfg(T=1 << 26), t=FAKE) == moe.MOE_ERR_BAD_SHAPE     # T * K reaches 2^32
    for kw in (dict(out_dtype=3), dict(out_dtype=-1)):
        assert call(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw


def test_linear_workspace():
    n = C.c_size_t(0)
    size = lambda c, g=0: moe.raw_call("moe_linear_mx4_workspace_size", c, g, C.byref(n))
    assert size(cfg(R=50, K=96)) == moe.MOE_OK and n.value == 2560 + 256
    assert size(cfg(R=5, K=96, T=100), 1) == moe.MOE_OK and n.value == 4864 + 512
    assert size(cfg(R=1, K=8224)) == moe.MOE_OK and n.value == 4352 + 512
    for kw in (dict(R=0), dict(R=0, T=5), dict(T=0), dict(R=1, K=8192), dict(R=1, K=96, T=50)):  # one row: no codes outside the kernel
        assert size(cfg(**kw), int("T" in kw)) == moe.MOE_OK and n.value == 0, kw
    assert size(None) == moe.MOE_ERR_NULL_ARG
    assert moe.raw_call("moe_linear_mx4_workspace_size", cfg(), 0, None) == moe.MOE_ERR_NULL_ARG
    for c, g in ((cfg(K=48), 0), (cfg(T=-1), 1), (cfg(), 2)):
        assert size(c, g) == moe.MOE_ERR_BAD_SHAPE
    assert size(cfg(R=50, K=96)) == moe.MOE_OK
    assert linear(cfg(R=50, K=96), nb=n.value - 1) == moe.MOE_ERR_WORKSPACE
    for kw in (dict(dtype=2), dict(dtype=-1)):
        assert linear(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED
    assert linear(cfg(), glu=2) == moe.MOE_ERR_UNSUPPORTED


def test_no_rows():
    assert mm(cfg(R=0), xq=None, xs=None, y=None) == moe.MOE_OK
    assert linear(cfg(R=0), x=None, y=None, work=None, nb=0) == moe.MOE_OK


def test_python_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    xq, xs, wq, ws = u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_quant_mx4(x)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_mm_mx4(xq, xs, wq, ws)
    for bad in ((x[0],), (x.float(),), (x.t(),)):
        with pytest.raises(ValueError):
            moe.moe_quant_mx4(*bad)
    with pytest.raises(ValueError, match="split"):
        moe.moe_quant_mx4(torch.zeros(2, 65, dtype=torch.bfloat16), swiglu=True)
    for bad in ((xq, xs, wq[None], ws[None]), (xq, xs, wq, ws[:, :1]), (xq, xs[:, :1], wq, ws), (xq.char(), xs, wq, ws),
                (xq[:, :16], xs, wq, ws)):
        with pytest.raises(ValueError):
            moe.moe_mm_mx4(*bad)
    with pytest.raises(ValueError, match="no gradient"):
        moe.moe_linear_mx4(x.clone().requires_grad_(), wq, ws)
    with pytest.raises(ValueError, match="no gradient"):
        moe.moe_quant_mx4(x.clone().requires_grad_())
    with pytest.raises(ValueError, match="no gradient"):
        moe.moe_mm_mx4(xq, xs, wq, ws, out=torch.zeros(4, 8, requires_grad=True))
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="forward-mode"):
            moe.moe_linear_mx4(dual, wq, ws)
