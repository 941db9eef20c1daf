"""Refusals of the few-token layer on 16-bit weights: every argument error is
found on the host, before anything is enqueued (no GPU needed)."""
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
    base = dict(T=4, H=64, I=32, E=8, topk=2, dtype=0)
    base.update(kw)
    return C.byref(moe.MoeFewCfg(*[base[n] for n, _ in moe.MoeFewCfg._fields_]))


def layer(c, x=FAKE, ids=FAKE, tw=FAKE, w1=FAKE, w2=FAKE, out=FAKE, ws=FAKE, nb=1 << 50):
    return moe.raw_call("moe_layer_mm", c, x, ids, tw, w1, w2, out, ws, nb, None)


def test_refusals():
    assert layer(None) == moe.MOE_ERR_NULL_ARG
    for n in ("x", "ids", "tw", "w1", "w2", "out", "ws"):
        assert layer(cfg(), **{n: None}) == moe.MOE_ERR_NULL_ARG, n
        assert layer(cfg(H=7), **{n: None}) == moe.MOE_ERR_NULL_ARG, n  # NULL comes before the shape
    for kw in (dict(T=-1), dict(H=0), dict(H=60), dict(I=0), dict(I=12), dict(E=0), dict(E=1025), dict(topk=0),
               dict(topk=33), dict(H=(1 << 16) + 8), dict(I=(1 << 16) + 8)):
        assert layer(cfg(**kw)) == moe.MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(T=65), dict(dtype=2), dict(dtype=-1)):
        assert layer(cfg(**kw)) == moe.MOE_ERR_UNSUPPORTED, kw
    for n in ("x", "w1", "w2", "out", "ws"):
        assert layer(cfg(), **{n: FAKE + 8}) == moe.MOE_ERR_MISALIGNED, n
    for n in ("ids", "tw"):
        assert layer(cfg(), **{n: FAKE + 2}) == moe.MOE_ERR_MISALIGNED, n
    assert layer(cfg(T=0), x=None, ids=None, tw=None, out=None, ws=None, nb=0) == moe.MOE_OK


def test_workspace():
    n = C.c_size_t(0)
    size = lambda c: moe.raw_call("moe_layer_mm_workspace_size", c, C.byref(n))
    assert size(cfg(T=0)) == moe.MOE_OK and n.value == 0
    assert size(cfg()) == moe.MOE_OK and n.value >= 4 * 2 * 32 * 4
    assert layer(cfg(), nb=n.value - 1) == moe.MOE_ERR_WORKSPACE
    assert size(None) == moe.MOE_ERR_NULL_ARG and moe.raw_call("moe_layer_mm_workspace_size", cfg(), None) == moe.MOE_ERR_NULL_ARG
    assert size(cfg(I=4)) == moe.MOE_ERR_BAD_SHAPE and size(cfg(T=65)) == moe.MOE_ERR_UNSUPPORTED


def test_python_refusals():
    bf = torch.bfloat16
    x, w1, w2 = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, 64, dtype=bf), torch.zeros(8, 64, 32, dtype=bf)
    ids, tw = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_layer_mm(x, ids, tw, w1, w2)
    for bad in ((x.half(), ids, tw, w1, w2), (x, ids.long(), tw, w1, w2), (x, ids[:2], tw, w1, w2), (x, ids, tw[:, :1], w1, w2),
                (x, ids, tw, w1[:, :63], w2), (x, ids, tw, w1[:4], w2), (x, ids, tw, w1, w2[:, :, :16]), (x[0], ids, tw, w1, w2)):
        with pytest.raises(ValueError):
            moe.moe_layer_mm(*bad)
    for k in (0, 2, 3, 4):
        args = [x, ids, tw, w1, w2]
        args[k] = args[k].clone().requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            moe.moe_layer_mm(*args)
