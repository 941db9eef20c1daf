"""The row-major products among other work of autograd's, of streams and of
threads (needs an MI355X)."""
import pytest
import torch

import bit_grouped_gemm_amd as moe
from test_gpu_mm import BF16, DEV, FP32, codes, gen, offs, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load()
    yield


def operands(seed=71, counts=(40, 0, 7, 130), N=136, K=256):
    g = gen(seed)
    E, R = len(counts), sum(counts)
    a = dict(x=rand(g, R, K), w=rand(g, E, N, K, scale=0.1), dy=rand(g, R, N), o=offs(list(counts)),
             wq=codes(g, E, N, K), ws=torch.rand(E, N, device=DEV, generator=g) * 1e-3)
    a["xq"], a["xs"] = moe.moe_quant_i8(a["x"])
    return a


# entry point -> (call into the caller's `out`, the result without one)
INTO = {
    "moe_grouped_mm": (lambda a, out: moe.moe_grouped_mm(a["x"], a["w"], a["o"], out=out),
                       lambda a: moe.moe_grouped_mm(a["x"], a["w"], a["o"])),
    "moe_grouped_mm_dgrad": (lambda a, out: moe.moe_grouped_mm_dgrad(a["dy"], a["w"], a["o"], out=out),
                             lambda a: moe.moe_grouped_mm_dgrad(a["dy"], a["w"], a["o"])),
    "moe_grouped_mm_wgrad": (lambda a, out: moe.moe_grouped_mm_wgrad(a["dy"], a["x"], a["o"], out=out),
                             lambda a: moe.moe_grouped_mm_wgrad(a["dy"], a["x"], a["o"])),
    "moe_mm_i8": (lambda a, out: moe.moe_mm_i8(a["xq"], a["xs"], a["wq"], a["ws"], a["o"], out=out),
                  lambda a: moe.moe_mm_i8(a["xq"], a["xs"], a["wq"], a["ws"], a["o"])),
    "moe_linear_i8": (lambda a, out: moe.moe_linear_i8(a["x"], a["wq"], a["ws"], a["o"], out=out),
                      lambda a: moe.moe_linear_i8(a["x"], a["wq"], a["ws"], a["o"])),
    "moe_quant_i8": (lambda a, out: moe.moe_quant_i8(a["x"], scales=out)[1], lambda a: moe.moe_quant_i8(a["x"])[1]),
}


@pytest.mark.parametrize("name", list(INTO))
def test_a_buffer_that_a_backward_pass_saved(name):
    """A buffer that is written again between a product that saved it and the
    backward pass: an error, as with PyTorch's own operations, not the gradient of the new values."""
    into, fresh = INTO[name]
    a, b = operands(), operands(seed=72)
    want = fresh(a)
    buf = torch.empty_like(want)
    p = torch.ones_like(want).requires_grad_()
    into(a, buf)
    (buf * p).sum().backward()
    assert torch.equal(p.grad, want)  # once written, read and done with
    loss = (into(a, buf) * p).sum()
    into(b, buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # a slice of it counts as well
    loss = (buf[:1] * p[:1]).sum()
    into(a, buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_buffers_of_inference_mode():
    a = operands()
    with torch.inference_mode():
        for into, fresh in INTO.values():
            want = fresh(a)
            buf = torch.zeros_like(want)
            assert torch.equal(into(a, buf), want)
    q = torch.zeros_like(a["xq"])
    version = q._version
    moe.moe_quant_i8(a["x"], codes=q)
    assert q._version > version and torch.equal(q, a["xq"])
