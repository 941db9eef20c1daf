"""The norm's gradients where hooks on saved tensors, as offloading and packing use
them, give back equal values in other places and orders of memory (needs an MI355X)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def unaligned(p):
    room = torch.empty(p.numel() + 1, dtype=p.dtype, device=p.device)
    room[1:] = p.reshape(-1)
    return room[1:].view(p.shape)


HOOKS = {
    "strides": (lambda t: t.detach().t().contiguous() if t.dim() == 2 else t.detach(),
                lambda p: p.t() if p.dim() == 2 else p),
    "alignment": (lambda t: t.detach(), unaligned),
    "host": (lambda t: t.detach().cpu(), lambda p: p.to(DEV)),
}


@pytest.mark.parametrize("hook", list(HOOKS))
@pytest.mark.parametrize("R,K,dtype,weight_dtype", [(6, 64, BF16, BF16), (33, 4096, FP16, FP32), (300, 1032, BF16, FP32)])
def test_hooks_on_saved_tensors(R, K, dtype, weight_dtype, hook):
    import bit_grouped_gemm_amd as moe
    print("test_hooks_on_saved_tensors", R, K, dtype, weight_dtype, hook, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(R + K)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
    x, res = rand(R, K).to(dtype).requires_grad_(), rand(R, K).to(dtype).requires_grad_()
    w = rand(K).to(weight_dtype).requires_grad_()
    dy, ds = rand(R, K).to(dtype), rand(R, K).to(dtype)

    def grads():
        y, s = moe.moe_rms_norm(x, w, res)
        alone = moe.moe_rms_norm(x, w)
        return lambda: (*torch.autograd.grad((y, s), (x, res, w), (dy, ds)), *torch.autograd.grad(alone, (x, w), dy))

    want = grads()()
    with torch.autograd.graph.saved_tensors_hooks(*HOOKS[hook]):
        back = grads()
    for a, b in zip(back(), want):
        assert a.is_contiguous() and torch.equal(a, b)
    assert all(t.abs().sum() > 0 for t in want)


def test_a_weight_with_other_data_is_refused():
    import bit_grouped_gemm_amd as moe
    x = torch.randn(4, 64, device=DEV).to(BF16)
    for other in (torch.ones(8, dtype=BF16, device=DEV), torch.ones(128, dtype=BF16, device=DEV)):
        w = torch.ones(64, dtype=BF16, device=DEV, requires_grad=True)
        y = moe.moe_rms_norm(x, w)
        w.data = other
        with pytest.raises(ValueError, match="weight"):
            torch.autograd.grad(y, w, torch.ones_like(y))


@pytest.mark.parametrize("R,K,dtype,weight_dtype", [(1, 8, BF16, BF16), (33, 4096, FP16, FP32), (300, 1032, BF16, FP32),
                                                    (5, 16384, FP16, FP16), (1003, 264, BF16, BF16)])
def test_the_entry_point_is_what_autograd_gives(R, K, dtype, weight_dtype):
    """moe_rms_norm_backward on the forward pass's own sum and rstd, bit for bit."""
    import bit_grouped_gemm_amd as moe
    print("test_the_entry_point_is_what_autograd_gives", R, K, dtype, weight_dtype, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(R + K)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
    x, res, w = rand(R, K).to(dtype).requires_grad_(), rand(R, K).to(dtype), rand(K).to(weight_dtype).requires_grad_()
    dy, ds = rand(R, K).to(dtype), rand(R, K).to(dtype)
    y, s = moe.moe_rms_norm(x, w, res, eps=1e-5)
    rstd = [t for t in y.grad_fn.saved_tensors if t.shape == (R,) and t.dtype == FP32][0]
    # 48 roundings, as rstd has fewer than y
    want = 1 / torch.sqrt(s.detach().double().square().mean(1) + 1e-5)
    assert ((rstd.double() - want).abs() <= 48 * 2.0 ** -24 * want).all()
    for d in (ds, None):
        dx, dw = torch.autograd.grad((y, s) if d is not None else y, (x, w), (dy, d) if d is not None else dy,
                                     retain_graph=True)
        for work in (None, torch.full((moe.moe_rms_norm_backward_workspace_size(R, K) + 64,), 255, dtype=torch.uint8, device=DEV)):
            a, b = moe.moe_rms_norm_backward(dy, d, s.detach(), rstd, w.detach(), eps=1e-5, work=work)
            assert torch.equal(a, dx) and torch.equal(b, dw)
