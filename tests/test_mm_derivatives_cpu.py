"""What the row-major products do with operands whose derivative they do not
give: refused before any pointer is taken, so no GPU is needed."""
import pytest
import torch
from torch.autograd import forward_ad

import bit_grouped_gemm_amd as moe

BF16, FP32, I8 = torch.bfloat16, torch.float32, torch.int8


def operands():
    z = torch.zeros
    return dict(x=z(4, 64, dtype=BF16), w=z(2, 32, 64, dtype=BF16), dy=z(4, 32, dtype=BF16), xs=z(4), ws=z(2, 32),
                xq=z(4, 64, dtype=I8), wq=z(2, 32, 64, dtype=I8), off=z(3, dtype=torch.int32), y=z(4, 32, dtype=BF16),
                dx=z(4, 64, dtype=BF16), dw=z(2, 32, 64, dtype=BF16), scales=z(4))


# entry point -> (the call, the operands whose derivative would be lost)
CALLS = {
    "moe_grouped_mm": (lambda a: moe.moe_grouped_mm(a["x"], a["w"], a["off"], out=a["y"]), ("y",)),
    "moe_grouped_mm_dgrad": (lambda a: moe.moe_grouped_mm_dgrad(a["dy"], a["w"], a["off"], out=a["dx"]),
                             ("dy", "w", "dx")),
    "moe_grouped_mm_wgrad": (lambda a: moe.moe_grouped_mm_wgrad(a["dy"], a["x"], a["off"], out=a["dw"]),
                             ("dy", "x", "dw")),
    "moe_quant_i8": (lambda a: moe.moe_quant_i8(a["x"], scales=a["scales"]), ("x", "scales")),
    "moe_mm_i8": (lambda a: moe.moe_mm_i8(a["xq"], a["xs"], a["wq"], a["ws"], a["off"], out=a["y"]),
                  ("xs", "ws", "y")),
    "moe_linear_i8": (lambda a: moe.moe_linear_i8(a["x"], a["wq"], a["ws"], a["off"], out=a["y"]), ("x", "ws", "y")),
}
EACH = [(name, which) for name, (_, some) in CALLS.items() for which in some]


@pytest.mark.parametrize("name,which", EACH)
def test_an_operand_that_needs_a_gradient_is_refused(name, which):
    a = operands()
    a[which].requires_grad_()
    with pytest.raises(ValueError, match="has no gradient"):
        CALLS[name][0](a)
    # where no graph is built, the call goes on to its other checks (these tensors are no GPU's)
    with torch.no_grad(), pytest.raises(ValueError, match="must live on the GPU"):
        CALLS[name][0](a)


@pytest.mark.parametrize("name,which", EACH + [("moe_grouped_mm", "x"), ("moe_grouped_mm", "w")])
def test_an_operand_with_a_tangent_is_refused(name, which):
    """A dual tensor does not say that it needs a gradient; no_grad leaves forward mode on."""
    a = operands()
    with forward_ad.dual_level():
        a[which] = forward_ad.make_dual(a[which], torch.ones_like(a[which]))
        assert not a[which].requires_grad
        for mode in (torch.enable_grad(), torch.no_grad()):
            with mode, pytest.raises(ValueError, match="no forward-mode derivative"):
                CALLS[name][0](a)
    # a level without a tangent is no reason to refuse
    with forward_ad.dual_level(), pytest.raises(ValueError, match="must live on the GPU"):
        CALLS[name][0](operands())


def test_a_differentiable_operand_with_a_tangent_is_refused():
    a = operands()
    with forward_ad.dual_level():
        x = forward_ad.make_dual(a["x"].requires_grad_(), torch.ones_like(a["x"]))
        with pytest.raises(ValueError, match="no forward-mode derivative"):
            moe.moe_grouped_mm(x, a["w"], a["off"])
