"""The row-major products among other work of autograd's, of streams and of
threads (needs an MI355X)."""
import threading

import pytest
import torch

import bit_grouped_gemm_amd as moe
from test_gpu_mm import BF16, DEV, codes, gen, offs, rand

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


def test_tensors_that_are_not_contiguous_are_refused():
    """Views with other strides, broadcast ones and slices of columns, for every operand and output."""
    a = operands()
    wide = lambda t: torch.cat([t, t], -1)[..., :t.shape[-1]]
    turned = lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2)
    calls = {"x": lambda b: moe.moe_grouped_mm(b["x"], b["w"], b["o"]),
             "w": lambda b: moe.moe_grouped_mm(b["x"], b["w"], b["o"]),
             "dy": lambda b: moe.moe_grouped_mm_dgrad(b["dy"], b["w"], b["o"]),
             "wq": lambda b: moe.moe_mm_i8(b["xq"], b["xs"], b["wq"], b["ws"], b["o"]),
             "ws": lambda b: moe.moe_linear_i8(b["x"], b["wq"], b["ws"], b["o"]),
             "xq": lambda b: moe.moe_mm_i8(b["xq"], b["xs"], b["wq"], b["ws"], b["o"])}
    for name, call in calls.items():
        call(a)
        for view in (wide, turned, lambda t: t[:1].expand_as(t)):
            with pytest.raises(ValueError, match="contiguous"):
                call({**a, name: view(a[name])})
    for name, view in (("o", torch.stack([a["o"], a["o"]], 1)[:, 0]), ("xs", torch.stack([a["xs"], a["xs"]], 1)[:, 0])):
        with pytest.raises(ValueError, match="contiguous"):
            moe.moe_mm_i8(a["xq"], view if name == "xs" else a["xs"], a["wq"], a["ws"], view if name == "o" else a["o"])
    for name, (into, fresh) in INTO.items():
        want = fresh(a)
        with pytest.raises(ValueError, match="contiguous"):
            into(a, torch.stack([want, want], -1)[..., 0])
    with pytest.raises(moe.MoeError):  # an address between two 16-byte steps
        moe.moe_grouped_mm(torch.empty(a["x"].numel() + 4, dtype=BF16, device=DEV)[4:].view_as(a["x"]), a["w"], a["o"])


# (PyTorch's remark that the leaves' gradients belong to another stream: that is what is tested)
@pytest.mark.filterwarnings("ignore:The AccumulateGrad node's stream")
def test_backward_on_another_stream_than_forward():
    """Forward on a side stream, behind work that delays it; the backward pass is asked for on the main one."""
    a = operands()
    want = (moe.moe_grouped_mm_dgrad(a["dy"], a["w"], a["o"]), moe.moe_grouped_mm_wgrad(a["dy"], a["x"], a["o"]))
    side = torch.cuda.Stream()
    big = torch.randn(2048, 2048, device=DEV)
    for _ in range(3):
        x, w = a["x"].clone().requires_grad_(), a["w"].clone().requires_grad_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                big = torch.tanh(big @ big)
            y = moe.moe_grouped_mm(x, w, a["o"])
        torch.cuda.current_stream().wait_stream(side)
        got = torch.autograd.grad(y, (x, w), a["dy"])
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        # the other way round
        y = moe.moe_grouped_mm(x, w, a["o"])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                big = torch.tanh(big @ big)
            got = torch.autograd.grad(y, (x, w), a["dy"])
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_calls_from_two_threads():
    """Each thread on its own stream with its own shapes, calls of both in flight: nothing is shared."""
    sets = [operands(81, (40, 0, 7, 130), 136, 256), operands(82, (1500, 300), 264, 128)]

    def everything(a):
        out = [fresh(a) for _, fresh in INTO.values()]
        x, w = a["x"].detach().clone().requires_grad_(), a["w"].detach().clone().requires_grad_()
        return out + list(torch.autograd.grad(moe.moe_grouped_mm(x, w, a["o"]), (x, w), a["dy"]))

    want = [everything(a) for a in sets]
    torch.cuda.synchronize()
    wrong, done = [], []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for n in range(20):
                for k, (p, q) in enumerate(zip(everything(sets[i]), want[i])):
                    if not torch.equal(p, q):
                        wrong.append((i, n, k))
        stream.synchronize()
        done.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(done) == [0, 1] and not wrong
