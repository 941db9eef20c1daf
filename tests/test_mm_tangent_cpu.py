"""A forward-mode tangent on the gradient that reaches moe_grouped_mm's backward pass is
refused, as on its operands: dx and dw would come back without it (no GPU needed, the
library calls are replaced by recorders)."""
import pytest
import torch
from torch.autograd import forward_ad

import bit_grouped_gemm_amd as moe

BF16 = torch.bfloat16


def test_incoming_gradient(monkeypatch):
    calls = []
    monkeypatch.setattr(moe, "_addr", lambda name, t, *rest: t.data_ptr() or None)
    monkeypatch.setattr(moe, "_call", lambda name, *rest: calls.append(name))
    x, w = torch.zeros(4, 64, dtype=BF16, requires_grad=True), torch.zeros(2, 8, 64, dtype=BF16, requires_grad=True)
    offsets = torch.tensor([0, 1, 4], dtype=torch.int32)
    one = torch.ones(4, 8, dtype=BF16)
    with forward_ad.dual_level():
        y = moe.moe_grouped_mm(x, w, offsets)
        calls.clear()
        with pytest.raises(ValueError, match="forward-mode"):
            torch.autograd.grad(y, (x, w), forward_ad.make_dual(one.clone(), one.clone()))
        assert not calls
        torch.autograd.grad(moe.moe_grouped_mm(x, w, offsets), (x, w), one)
        assert calls == ["moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad"]
