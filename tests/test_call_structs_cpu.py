"""The calls' structs are kept by their values: a number that is handed over as a
tensor counts as it is at the call, and one that no 32-bit field holds is refused
(no GPU needed: the library calls are replaced by recorders)."""
import pytest
import torch

import bit_grouped_gemm_amd as moe

BF16 = torch.bfloat16


@pytest.fixture
def structs(monkeypatch):
    seen = []
    monkeypatch.setattr(moe, "_addr", lambda name, t, *rest: t.data_ptr() or None)
    monkeypatch.setattr(moe, "_call", lambda name, index, c, *rest: seen.append(
        {n: getattr(c._obj, n) for n, _ in c._obj._fields_}))
    return seen


def operands():
    return torch.zeros(4, 256, dtype=BF16), torch.ones(256, dtype=BF16)


def test_an_eps_tensor_that_changes(structs):
    x, w = operands()
    eps = torch.tensor(1e-3)
    rstd = torch.ones(4)
    calls = (lambda: moe.moe_rms_norm(x, w, eps=eps), lambda: moe.moe_rms_norm_quant(x, w, eps=eps),
             lambda: moe.moe_rms_norm_backward(x, None, x, rstd, w, eps=eps),
             lambda: moe.moe_rms_norm(x, w.clone().requires_grad_(), eps=eps))
    for call in calls:
        for value in (2.0 ** -10, 2.0 ** -7):
            eps.fill_(value)
            call()
            assert structs.pop()["eps"] == value and not structs


def test_the_backward_pass_has_the_eps_of_its_forward_pass(structs):
    x, w = operands()
    w.requires_grad_()
    eps = torch.tensor(2.0 ** -10)
    y = moe.moe_rms_norm(x, w, eps=eps)
    eps.fill_(0.5)
    y.sum().backward()
    assert [s["eps"] for s in structs] == [2.0 ** -10] * 2


def test_a_group_tensor_that_changes(structs):
    x, w = operands()
    group, fmt = torch.tensor(32), torch.tensor(moe.QFMT_E4M3)
    for value in (32, 128):
        group.fill_(value)
        _, scales, _, _ = moe.moe_rms_norm_quant(x, w, group=group, fmt=fmt)
        assert scales.shape == (4, 256 // value) and structs.pop()["group"] == value
    fmt.fill_(moe.QFMT_I8)
    codes, scales, _, _ = moe.moe_rms_norm_quant(x, w, group=group, fmt=fmt)
    assert structs.pop()["fmt"] == moe.QFMT_I8 and codes.dtype == torch.int8 and scales.shape == (4,)


@pytest.mark.parametrize("kw", [dict(group=(1 << 32) + 32), dict(group=32 - (1 << 32)), dict(fmt=1 << 32),
                                dict(fmt=(1 << 32) + 2), dict(fmt=2 - (1 << 32))], ids=str)
def test_numbers_past_32_bits(structs, kw):
    x, w = operands()
    with pytest.raises(ValueError, match="32 bits"):
        moe.moe_rms_norm_quant(x, w, **kw)
    assert not structs


@pytest.mark.parametrize("value", [1.5, "128", None])
def test_numbers_that_are_no_integers(structs, value):
    x, w = operands()
    moe.moe_rms_norm_quant(x, w, group=128)
    structs.clear()
    for kw in (dict(group=value), dict(fmt=value)):
        with pytest.raises(TypeError):
            moe.moe_rms_norm_quant(x, w, **kw)
    assert not structs


def test_sizes_past_32_bits():
    far = (1 << 32) + 5
    for call in (lambda: moe.moe_linear_mx4_workspace_size(far, 64), lambda: moe.moe_linear_mx4_workspace_size(5, 64, far),
                 lambda: moe.moe_linear_mx4_workspace_size(5, far + 59),
                 lambda: moe.moe_layer_mm_workspace_size(far, 64, 64, 8, 2),
                 lambda: moe.moe_rms_norm_backward_workspace_size(far, 64),
                 lambda: moe.moe_rms_norm_backward_workspace_size(5, far + 59)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_a_size_tensor_that_changes():
    n = torch.tensor(5)
    for size in (lambda: moe.moe_linear_mx4_workspace_size(n, 64), lambda: moe.moe_linear_mx4_workspace_size(7, 64, n),
                 lambda: moe.moe_layer_mm_workspace_size(n, 64, 64, 8, 2),
                 lambda: moe.moe_rms_norm_backward_workspace_size(n, 64)):
        got = []
        for value in (5, 60, 5):
            n.fill_(value)
            got.append(size())
        assert got[0] == got[2]
    n.fill_(5)
    few = moe.moe_linear_mx4_workspace_size(n, 64)
    n.fill_(50)
    assert moe.moe_linear_mx4_workspace_size(n, 64) == moe.moe_linear_mx4_workspace_size(50, 64) > few
