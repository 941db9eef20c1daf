"""A forward-mode tangent on what reaches the norm's backward pass is refused, as
on its operands: the gradients would come back without it (no GPU needed, the
library calls are replaced by recorders)."""
import pytest
import torch
from torch.autograd import forward_ad

import bit_grouped_gemm_amd as moe

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(moe, "_addr", lambda name, t, *rest: t.data_ptr() or None)
    monkeypatch.setattr(moe, "_call", lambda name, *rest: seen.append(name))
    return seen


@pytest.mark.parametrize("which", ["dy", "ds"])
def test_incoming_gradients(calls, which):
    x, w, res = (torch.zeros(4, 64, dtype=BF16, requires_grad=True), torch.ones(64, dtype=BF16, requires_grad=True),
                 torch.zeros(4, 64, dtype=BF16))
    one = torch.ones(4, 64, dtype=BF16)
    y, s = moe.moe_rms_norm(x, w, res)
    calls.clear()
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(one.clone(), one.clone())
        with pytest.raises(ValueError, match="forward-mode"):
            torch.autograd.grad((y, s), (x, w), (dual, one) if which == "dy" else (one, dual))
        assert not calls
        # one without a tangent is none of its business, nor is the sum's gradient alone, which passes through
        y, s = moe.moe_rms_norm(x, w, res)
        torch.autograd.grad((y, s), (x, w), (one, one))
        assert calls == ["moe_rms_norm", "moe_rms_norm_backward"]
        y, s = moe.moe_rms_norm(x, w, res)
        (dx,) = torch.autograd.grad(s, x, dual)
        assert torch.equal(forward_ad.unpack_dual(dx).tangent, one)

