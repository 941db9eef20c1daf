"""What the norm's backward pass takes back from autograd: hooks on saved tensors
and leaves with other data may have made something else of it.  The library call is
replaced by a recorder, so all of this runs without a GPU."""
import ctypes as C

import pytest
import torch

import bit_grouped_gemm_amd as moe

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
R, K = 6, 64



class Calls(list):
    look = True  # whether the memory at the addresses is read and written


@pytest.fixture
def calls(monkeypatch):
    """The backward calls, each with the rows found at the addresses it was given."""
    seen = Calls()

    def rms_norm(x, weight, residual, eps, out=None, sum_out=None, want_rstd=False):
        s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
        rstd = 1 / torch.sqrt(s.float().square().mean(1) + eps)
        return (s.float() * rstd[:, None] * weight.float()).to(x.dtype), None if residual is None else s, rstd

    def call(name, index, cfg, dy, ds, s, rstd, weight, dx, dw, work, need):
        def rows(address, n, kind):
            assert address is None or address % 16 == 0
            return None if address is None else torch.frombuffer((C.c_char * (n * kind.itemsize)).from_address(address),
                                                                 dtype=kind).clone()
        if not seen.look:
            return seen.append(name)
        c = cfg._obj
        ty = {0: BF16, 1: FP16, 2: FP32}
        n = c.R * c.K
        seen.append(dict(name=name, R=c.R, K=c.K, dy=rows(dy, n, ty[c.dtype]), ds=rows(ds, n, ty[c.dtype]),
                         s=rows(s, n, ty[c.dtype]), rstd=rows(rstd, c.R, FP32),
                         weight=rows(weight, c.K, ty[c.weight_dtype])))
        for address, size in ((dx, n * ty[c.dtype].itemsize), (dw, c.K * ty[c.weight_dtype].itemsize)):
            if address is not None:
                C.memset(address, 0, size)

    monkeypatch.setattr(moe, "_rms_norm", rms_norm)
    monkeypatch.setattr(moe, "_call", call)
    return seen


def operands(residual, weight_dtype=BF16):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(R, K, generator=g).to(BF16).requires_grad_()
    w = torch.randn(K, generator=g).to(weight_dtype).requires_grad_()
    res = torch.randn(R, K, generator=g).to(BF16) if residual else None
    return x, w, res, torch.randn(R, K, generator=g).to(BF16)


def first(y):
    return y[0] if isinstance(y, tuple) else y


@pytest.mark.parametrize("residual", [False, True])
def test_saved_rows_with_other_strides(calls, residual):
    """A hook that gives back equal values in another order of memory: the call sees rows."""
    x, w, res, dy = operands(residual)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().t().contiguous() if t.dim() == 2 else t.detach(),
                                                  lambda p: p.t() if p.dim() == 2 else p):
        y = moe.moe_rms_norm(x, w, res)
    dx, dw = torch.autograd.grad(first(y), (x, w), dy)
    (c,) = calls
    s = x.detach() if res is None else (x.detach().float() + res.float()).to(BF16)
    assert torch.equal(c["s"].view(R, K), s) and torch.equal(c["dy"].view(R, K), dy)
    assert torch.equal(c["weight"], w.detach())
    assert dx.is_contiguous() and dw.is_contiguous()


def test_saved_tensors_that_are_unaligned(calls):
    """A hook that packs into one buffer: views two bytes off are moved."""
    def unpack(p):
        room = torch.empty(p.numel() + 1, dtype=p.dtype)
        room[1:] = p.reshape(-1)
        return room[1:].view(p.shape)
    x, w, res, dy = operands(True)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(), unpack):
        y, s = moe.moe_rms_norm(x, w, res)
    torch.autograd.grad(y, (x, w), dy)
    (c,) = calls
    assert torch.equal(c["s"].view(R, K), s.detach()) and torch.equal(c["weight"], w.detach())


OTHERS = {
    "smaller": lambda t: t[..., :8].clone(),
    "larger": lambda t: torch.cat([t, t], -1),
    "other_type": lambda t: t.to(FP16),
    "other_device": lambda t: t.to("meta"),
    "fewer_dimensions": lambda t: t.reshape(-1)[0],
}


@pytest.mark.parametrize("which", ["x", "weight"])
@pytest.mark.parametrize("other", list(OTHERS))
def test_a_leaf_with_other_data(calls, which, other):
    calls.look = False
    x, w, _, dy = operands(False)
    y = moe.moe_rms_norm(x, w)
    leaf = x if which == "x" else w
    if other == "other_device":
        return by_hook(calls, which, other)  # (.data keeps the device's kind)
    if other == "other_type":
        leaf.data = leaf.data.to(FP16)
    else:
        leaf.data = OTHERS[other](leaf.data)
    with pytest.raises((ValueError, RuntimeError)):
        torch.autograd.grad(y, (x, w), dy)
    assert not calls


def by_hook(calls, which, other):
    calls.look = False
    x, w, _, dy = operands(False)
    dims = {"x": 2, "weight": 1}[which]
    other = OTHERS[other]
    with torch.autograd.graph.saved_tensors_hooks(
            lambda t: t.detach(), lambda p: other(p) if p.dim() == dims and p.dtype != FP32 else p):
        y = moe.moe_rms_norm(x, w)
    with pytest.raises(ValueError, match="weight" if which == "weight" else "sum"):
        torch.autograd.grad(y, (x, w), dy)
    assert not calls


@pytest.mark.parametrize("which", ["x", "weight"])
@pytest.mark.parametrize("other", list(OTHERS))
def test_a_hook_that_gives_back_something_else(calls, which, other):
    by_hook(calls, which, other)


@pytest.mark.parametrize("other", ["shorter", "other_type"])
def test_a_hook_on_rstd(calls, other):
    calls.look = False
    x, w, _, dy = operands(False)
    change = (lambda p: p[:2]) if other == "shorter" else (lambda p: p.double())
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach(), lambda p: change(p) if p.dtype == FP32 else p):
        y = moe.moe_rms_norm(x, w)
    with pytest.raises(ValueError, match="rstd"):
        torch.autograd.grad(y, (x, w), dy)
    assert not calls


def test_a_function_hook_that_changes_the_gradient(calls):
    calls.look = False
    x, w, _, dy = operands(False)
    for change in (lambda g: (g[0][:2],), lambda g: (g[0].half(),), lambda g: (g[0].to("meta"),)):
        y = moe.moe_rms_norm(x, w)
        y.grad_fn.register_prehook(change)
        with pytest.raises((ValueError, RuntimeError)):
            torch.autograd.grad(y, (x, w), dy)
    assert not calls


def test_the_ordinary_call_is_one(calls):
    for weight_dtype in (BF16, FP32):
        for residual in (False, True):
            x, w, res, dy = operands(residual, weight_dtype)
            y = moe.moe_rms_norm(x, w, res)
            dx, dw = torch.autograd.grad(first(y), (x, w), dy)
            assert dx.dtype == BF16 and dw.dtype == weight_dtype and dx.shape == (R, K) and dw.shape == (K,)
            c = calls.pop()
            assert not calls and (c["R"], c["K"]) == (R, K) and c["name"] == "moe_rms_norm_backward"
