"""The row-major products and the int8 quantiser against plain 64-bit forms
(needs an MI355X).

Tolerances.  A product of 16-bit values is exact in fp32, and K of them summed
in fp32 in any order are off by at most K 2^-23 sum |x w| (2^-23 rather than
2^-24 per addition also covers an adder that truncates); the one rounding to the
output type adds eps / 2 of the value (fp16: or half its smallest subnormal, 2^-25).  An int8 product's sum
is exact; turning it to fp32 and the two scalings round three times (2^-24
each), then the output type's rounding.
"""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M().load()
    yield


def M():
    import bit_grouped_gemm_amd as moe
    return moe


def note(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rand(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


def offs(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 * 1.01


def near(got, ref, mag, terms, what):
    """|got - ref| within the sum's error and the output's rounding."""
    tol = (terms + 8) * 2.0 ** -23 * mag + half_step(got.dtype) * ref.abs()
    tol = tol * 1.01 + (2.0 ** -25 if got.dtype == FP16 else 1e-38)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, (what, worst, err.max().item())


def ref_fwd(x, w, o):
    R, N = x.shape[0], w.shape[1]
    y = torch.zeros(R, N, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(o[e]), int(o[e + 1])
        we = w[e].double().t()
        y[a:b] = x[a:b].double() @ we
        mag[a:b] = x[a:b].double().abs() @ we.abs()
    return y, mag


def ref_wgrad(dy, x, o):
    E = o.numel() - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(dw)
    for e in range(E):
        a, b = int(o[e]), int(o[e + 1])
        d = dy[a:b].double().t()
        dw[e] = d @ x[a:b].double()
        mag[e] = d.abs() @ x[a:b].double().abs()
    return dw, mag


# (rows per group, rows behind the last group, N, K)
SHAPES = {
    "one_row": ([1], 0, 8, 8),
    "one_row_of_many": ([0, 0, 1, 0], 0, 128, 256),
    "tiny_layer": ([5, 0, 7, 1, 3, 0, 13, 8], 0, 128, 256),
    "no_full_tile": ([3, 17, 64, 65], 0, 136, 200),
    "k_past_a_step": ([9, 33], 0, 264, 72),
    "behind_the_last": ([4, 0, 70], 31, 72, 136),
    "only_behind": ([0, 0, 0], 77, 264, 64),
    "first_and_last_empty": ([0, 100, 129, 0], 3, 520, 1000),
    "about_128_a_group": ([127, 128, 129, 0, 200], 0, 392, 328),
    "large_groups": ([511, 0, 700, 257], 65, 264, 456),
    "one_large_group": ([1025], 0, 1032, 520),
    "skewed": ([900] + [0] * 30 + [1], 0, 256, 128),
    "many_groups": ([i % 5 for i in range(200)], 9, 64, 64),
    "most_groups": ([i % 3 for i in range(1024)], 5, 16, 32),
    "many_large_groups": ([257, 300, 0] * 45, 0, 72, 80),
    "long_k": ([2, 30], 0, 16, 8200),
    "rows_split_for_dw": ([3000, 0, 1511], 70, 72, 136),
    "rows_split_for_one_dw": ([33001], 0, 136, 264),
    "decode_slice": ([1, 0, 2, 1, 0, 0, 3, 1], 0, 1536, 4096),
}


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_products(name, dtype):
    moe = M()
    counts, tail, N, K = SHAPES[name]
    note("test_products", name, dtype)
    g = gen(hash((N, K)) % 1000)
    o = offs(counts)
    R, E, rows = sum(counts) + tail, len(counts), sum(counts)
    x, w, dy = rand(g, R, K, dtype=dtype), rand(g, E, N, K, dtype=dtype, scale=0.05), rand(g, R, N, dtype=dtype)
    y, mag = ref_fwd(x, w, o)
    for od in (dtype, FP32):
        got = moe.moe_grouped_mm(x, w, o, out_dtype=od)
        assert got.dtype == od
        near(got, y, mag, K, "y")
        assert not got[rows:].any()
        got = moe.moe_grouped_mm_dgrad(dy, w, o, out_dtype=od)
        dx, m = ref_fwd(dy, w.transpose(1, 2).contiguous(), o)
        near(got, dx, m, N, "dx")
        assert not got[rows:].any()
        got = moe.moe_grouped_mm_wgrad(dy, x, o, out_dtype=od)
        dw, m = ref_wgrad(dy, x, o)
        near(got, dw, m, max(counts), "dw")
        for e, n in enumerate(counts):
            assert n or not got[e].any()


def test_a_caller_s_rows_behind_the_last_group_stay():
    moe = M()
    g = gen(5)
    counts, tail, N, K = [3, 0, 70], 40, 264, 128
    o, R, rows = offs(counts), 113, 73
    x, w, dy = rand(g, R, K), rand(g, 3, N, K), rand(g, R, N)
    out, dx = torch.full((R, N), 7.0, dtype=BF16, device=DEV), torch.full((R, K), -3.0, dtype=BF16, device=DEV)
    moe.moe_grouped_mm(x, w, o, out=out)
    moe.moe_grouped_mm_dgrad(dy, w, o, out=dx)
    assert (out[rows:] == 7).all() and (dx[rows:] == -3).all()
    assert torch.equal(out[:rows], moe.moe_grouped_mm(x, w, o)[:rows])
    assert torch.equal(dx[:rows], moe.moe_grouped_mm_dgrad(dy, w, o)[:rows])
    dw = torch.full((3, N, K), 9.0, dtype=FP32, device=DEV)
    moe.moe_grouped_mm_wgrad(dy, x, o, out=dw)
    assert torch.equal(dw, moe.moe_grouped_mm_wgrad(dy, x, o, out_dtype=FP32))


@pytest.mark.parametrize("counts", [[5, 3, 6], [130, 70, 150], [600, 500, 700]], ids=["small", "middle", "large"])
def test_what_is_not_finite_stays_in_its_group(counts):
    """NaN and infinities of one group (and behind the last) reach no row of another, nor its gradient."""
    moe = M()
    g = gen(7)
    N, K = 72, 104
    o, R = offs(counts), sum(counts) + 20
    x, w, dy = rand(g, R, K), rand(g, 3, N, K), rand(g, R, N)
    clean = [moe.moe_grouped_mm(x, w, o), moe.moe_grouped_mm_dgrad(dy, w, o), moe.moe_grouped_mm_wgrad(dy, x, o)]
    a, b = counts[0], counts[0] + counts[1]
    for t in (x, dy):
        t[a:b] = float("nan")
        t[a + 1] = float("inf")
        t[sum(counts):] = float("nan")
    w[1] = float("nan")
    y, dx, dw = moe.moe_grouped_mm(x, w, o), moe.moe_grouped_mm_dgrad(dy, w, o), moe.moe_grouped_mm_wgrad(dy, x, o)
    rows = sum(counts)
    for got, want in ((y, clean[0]), (dx, clean[1])):
        assert torch.equal(got[:a], want[:a]) and torch.equal(got[b:rows], want[b:rows])
        assert torch.isnan(got[a:b]).all() and not got[rows:].any()
    assert torch.equal(dw[0], clean[2][0]) and torch.equal(dw[2], clean[2][2]) and torch.isnan(dw[1]).all()


def test_no_rows():
    moe = M()
    o = offs([0, 0])
    x, w, dy = rand(gen(1), 0, 64), rand(gen(1), 2, 32, 64), rand(gen(1), 0, 32)
    assert moe.moe_grouped_mm(x, w, o).shape == (0, 32)
    assert moe.moe_grouped_mm_dgrad(dy, w, o).shape == (0, 64)
    dw = moe.moe_grouped_mm_wgrad(dy, x, o)
    assert dw.shape == (2, 32, 64) and not dw.any()
    q, s = moe.moe_quant_i8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    wq, ws = torch.zeros(2, 32, 64, dtype=torch.int8, device=DEV), torch.ones(2, 32, device=DEV)
    assert moe.moe_mm_i8(q, s, wq, ws, o).shape == (0, 32)
    assert moe.moe_linear_i8(x, wq, ws, o).shape == (0, 32)
    # tokens, but none with a row
    t = torch.empty(0, dtype=torch.int32, device=DEV)
    assert moe.moe_linear_i8(rand(gen(1), 4, 64), wq, ws, o, row_token=t).shape == (0, 32)


@pytest.mark.parametrize("counts", [[5, 3, 6, 2], [130, 70, 150, 60], [600, 500, 700, 40]], ids=["small", "middle", "large"])
def test_a_run_of_the_groups(counts):
    """Some of the experts with their slice of the offsets: rows of the others, before and behind, belong to none."""
    moe = M()
    g = gen(9)
    N, K = 72, 112
    o, R = offs(counts), sum(counts) + 7
    x, w, dy = rand(g, R, K), rand(g, 4, N, K), rand(g, R, N)
    a, b = int(o[1]), int(o[3])
    part, wp = o[1:4], w[1:3].contiguous()
    for full, some, out in ((moe.moe_grouped_mm(x, w, o), lambda **k: moe.moe_grouped_mm(x, wp, part, **k), N),
                            (moe.moe_grouped_mm_dgrad(dy, w, o), lambda **k: moe.moe_grouped_mm_dgrad(dy, wp, part, **k), K)):
        got = some()
        assert torch.equal(got[a:b], full[a:b]) and not got[:a].any() and not got[b:].any()
        keep = torch.full((R, out), 7.0, dtype=BF16, device=DEV)
        some(out=keep)
        assert torch.equal(keep[a:b], full[a:b]) and (keep[:a] == 7).all() and (keep[b:] == 7).all()
    assert torch.equal(moe.moe_grouped_mm_wgrad(dy, x, part), moe.moe_grouped_mm_wgrad(dy, x, o)[1:3])
    wq, ws = codes(g, 4, N, K), torch.rand(4, N, device=DEV, generator=g)
    full = moe.moe_linear_i8(x, wq, ws, o)
    got = moe.moe_linear_i8(x, wq[1:3].contiguous(), ws[1:3].contiguous(), part)
    assert torch.equal(got[a:b], full[a:b]) and not got[:a].any() and not got[b:].any()


def test_wrong_offsets_stay_inside_the_tensors():
    """Offsets are clamped to the rows: rows that a wrong array does name come out right, nothing else is touched."""
    moe = M()
    g = gen(11)
    x, w = rand(g, 50, 64), rand(g, 2, 72, 64)
    o = torch.tensor([0, 20, 1 << 30], dtype=torch.int32, device=DEV)
    y, mag = ref_fwd(x, w, torch.tensor([0, 20, 50]))
    near(moe.moe_grouped_mm(x, w, o), y, mag, 64, "y")
    guard = torch.full((60, 72), 5.0, dtype=BF16, device=DEV)
    moe.moe_grouped_mm(x, w, torch.tensor([-7, 90, 20], dtype=torch.int32, device=DEV), out=guard[:50])
    assert (guard[50:] == 5).all()


def test_rows_past_32_bits():
    """R * K past 2^32 elements: the last rows of the operands and of the gradients."""
    moe = M()
    g = gen(13)
    R, K, N = (1 << 20) + 37, 4096, 64
    x = torch.zeros(R, K, dtype=BF16, device=DEV)
    x[-300:] = rand(g, 300, K)
    w = rand(g, 2, N, K)
    o = torch.tensor([0, R - 200, R], dtype=torch.int32, device=DEV)
    y = moe.moe_grouped_mm(x, w, o)
    ref, mag = ref_fwd(x[-300:], w, torch.tensor([0, 100, 300]))
    near(y[-300:], ref, mag, K, "y")
    assert not y[:-300].any()
    dy = torch.zeros(R, N, dtype=BF16, device=DEV)
    dy[-300:] = rand(g, 300, N)
    dx = moe.moe_grouped_mm_dgrad(dy, w, o)
    ref, mag = ref_fwd(dy[-300:], w.transpose(1, 2).contiguous(), torch.tensor([0, 100, 300]))
    near(dx[-300:], ref, mag, N, "dx")
    assert not dx[-1000:-300].any()
    dw = moe.moe_grouped_mm_wgrad(dy, x, o)
    ref, mag = ref_wgrad(dy[-300:], x[-300:], torch.tensor([0, 100, 300]))
    near(dw, ref, mag, 300, "dw")


def test_int8_rows_past_32_bits():
    """R * K past 2^31 codes, and past 2^32 bytes of activations."""
    moe = M()
    g = gen(14)
    R, K, N = (1 << 18) + 21, 8704, 72
    x = torch.zeros(R, K, dtype=BF16, device=DEV)
    x[-70:] = rand(g, 70, K)
    q, s = moe.moe_quant_i8(x)
    want = moe.moe_quant_i8(x[-70:].contiguous())
    assert torch.equal(q[-70:], want[0]) and torch.equal(s[-70:], want[1]) and not q[:-70].any()
    wq, ws = codes(g, N, K), torch.rand(N, device=DEV, generator=g) * 1e-3
    y = moe.moe_mm_i8(q, s, wq, ws, out_dtype=FP32)
    near_i8(y[-70:], (want[0].double() @ wq.double().t()) * want[1].double()[:, None] * ws.double(), "last rows")
    assert not y[:-70].any()


# ------------------------------------------------------------------ autograd
@pytest.mark.parametrize("out", [BF16, FP16, FP32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("E,N,K,rows", [(40, 776, 520, 20), (300, 264, 264, 9), (530, 8, 8, 3), (70, 1032, 264, 130),
                                        (30, 2056, 264, 300), (3, 520, 776, 1500), (1, 520, 520, 4000)],
                         ids=lambda v: str(v))
def test_wgrad_many_tiles(E, N, K, rows, out):
    """More tiles than CUs, with short reductions (one workgroup takes several
    tiles) and long ones, tile counts that no power of two divides, empty and
    long groups in between; and fewer tiles, whose rows are split."""
    g = gen(77)
    counts = [0 if E > 1 and e % 5 == 2 else rows * (3 if e % 7 == 3 else 1) - e % 3 for e in range(E)]
    o, R = offs(counts), sum(counts)
    dtype = FP16 if out == FP16 else BF16
    dy, x = rand(g, R, N, dtype=dtype), rand(g, R, K, dtype=dtype)
    ref, mag = ref_wgrad(dy, x, o)
    dw = torch.full((E, N, K), float("nan"), dtype=out, device=DEV)
    note(E, N, K, R, out)
    for _ in range(3):
        dw.fill_(float("nan"))
        M().moe_grouped_mm_wgrad(dy, x, o, out=dw)
        near(dw, ref, mag, max(counts), "dW")
    assert torch.equal(dw, M().moe_grouped_mm_wgrad(dy, x, o, out=torch.empty_like(dw)))


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_autograd_equals_the_gradient_products(dtype):
    moe = M()
    g = gen(17)
    counts, N, K = [40, 0, 7, 130], 136, 264
    o, R = offs(counts), 177 + 5
    x, w = rand(g, R, K, dtype=dtype).requires_grad_(), rand(g, 4, N, K, dtype=dtype).requires_grad_()
    dy = rand(g, R, N, dtype=dtype)
    y = moe.moe_grouped_mm(x, w, o)
    assert torch.equal(y, moe.moe_grouped_mm(x.detach(), w.detach(), o))
    y.backward(dy)
    assert torch.equal(x.grad, moe.moe_grouped_mm_dgrad(dy, w.detach(), o))
    assert torch.equal(w.grad, moe.moe_grouped_mm_wgrad(dy, x.detach(), o))
    assert not x.grad[177:].any()
    # a gradient that is broadcast, and one leaf alone
    x2 = x.detach().clone().requires_grad_()
    moe.moe_grouped_mm(x2, w.detach(), o).sum().backward()
    assert torch.equal(x2.grad, moe.moe_grouped_mm_dgrad(torch.ones_like(y), w.detach(), o))
    # a gradient that is a view at an odd place
    x3 = x.detach().clone().requires_grad_()
    flat = torch.empty(y.numel() + 4, dtype=dtype, device=DEV)[4:].view_as(y).copy_(dy)
    assert torch.equal(torch.autograd.grad(moe.moe_grouped_mm(x3, w.detach(), o), x3, flat)[0], x.grad)
    # the weights used twice: their gradients add up
    w2 = w.detach().clone().requires_grad_()
    (moe.moe_grouped_mm(x.detach(), w2, o) + moe.moe_grouped_mm(x.detach(), w2, o)).backward(dy)
    once = moe.moe_grouped_mm_wgrad(dy, x.detach(), o)
    assert torch.equal(w2.grad, once + once)
    with torch.no_grad():
        assert not moe.moe_grouped_mm(x, w, o).requires_grad
    # once differentiable: a gradient of the gradient is refused, not wrong
    g1, = torch.autograd.grad(moe.moe_grouped_mm(x, w, o).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g1.float().sum(), w)


def test_gradients_against_differences():
    """The product is linear in x and in w, so a difference of any length is the
    derivative: <dy, f(x + d) - f(x)> = <dx, d>.  All values are multiples of
    1/16 that stay small, so that every product and sum is exact in fp32."""
    moe = M()
    g = gen(19)
    counts, N, K = [33, 0, 90], 72, 136
    o, R = offs(counts), 123
    small = lambda *s: (torch.randint(-8, 9, s, device=DEV, generator=g) / 16).to(BF16)
    x, w, dy, d, dv = small(R, K), small(3, N, K), small(R, N), small(R, K), small(3, N, K)
    f = lambda a, b: moe.moe_grouped_mm(a, b, o, out_dtype=FP32).double()
    dx = moe.moe_grouped_mm_dgrad(dy, w, o, out_dtype=FP32).double()
    dw = moe.moe_grouped_mm_wgrad(dy, x, o, out_dtype=FP32).double()
    assert ((f(x + d, w) - f(x, w)) * dy.double()).sum().item() == (dx * d.double()).sum().item()
    assert ((f(x, w + dv) - f(x, w)) * dy.double()).sum().item() == (dw * dv.double()).sum().item()


# ------------------------------------------------------------------ int8
def codes(g, *shape):
    return torch.randint(-127, 128, shape, device=DEV, generator=g).to(torch.int8)


def near_i8(got, ref, what):
    tol = (3 * 2.0 ** -24 + half_step(got.dtype)) * 1.01 * ref.abs() + (2.0 ** -25 if got.dtype == FP16 else 1e-38)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), (what, (err - tol).max().item())


I8_SHAPES = {n: v for n, v in SHAPES.items() if v[3] % 16 == 0}
I8_SHAPES["k_of_16"] = ([1, 4], 0, 8, 16)
I8_SHAPES["k_past_a_step_i8"] = ([9, 70], 2, 264, 144)


@pytest.mark.parametrize("od", [BF16, FP16, FP32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name", list(I8_SHAPES))
def test_mm_i8_grouped(name, od):
    moe = M()
    counts, tail, N, K = I8_SHAPES[name]
    note("test_mm_i8_grouped", name, od)
    g = gen(23)
    o, rows = offs(counts), sum(counts)
    R, E = rows + tail, len(counts)
    T = max(1, R // 3)
    wq, ws = codes(g, E, N, K), torch.rand(E, N, device=DEV, generator=g) * 1e-3 + 1e-5
    # identity rows
    xq, xs = codes(g, R, K), torch.rand(R, device=DEV, generator=g) * 1e-2 + 1e-4
    e_of = torch.repeat_interleave(torch.arange(E, device=DEV), torch.tensor(counts, device=DEV))

    def ref(q, s):
        acc = torch.zeros(R, N, dtype=torch.float64, device=DEV)
        for e in range(E):
            a, b = int(o[e]), int(o[e + 1])
            acc[a:b] = q[a:b].double() @ wq[e].double().t()
        acc[:rows] *= s[:rows, None].double() * ws[e_of].double()
        return acc

    near_i8(moe.moe_mm_i8(xq, xs, wq, ws, o, out_dtype=od), ref(xq, xs), "identity")
    # gathered rows, two of them naming no token
    xq, xs = codes(g, T, K), torch.rand(T, device=DEV, generator=g) * 1e-2 + 1e-4
    t = torch.randint(0, T, (R,), device=DEV, generator=g).to(torch.int32)
    t[rows:] = -1
    if rows > 3:
        t[1], t[rows - 1] = -1, T
    ok = ((t >= 0) & (t < T))
    q = xq[t.long().clamp(0, T - 1)] * ok[:, None].to(torch.int8)
    s = xs[t.long().clamp(0, T - 1)]
    got = moe.moe_mm_i8(xq, xs, wq, ws, o, row_token=t, out_dtype=od)
    near_i8(got, ref(q, s), "gathered")
    assert not got[rows:].any() and not got[~ok].any()
    keep = torch.full((R, N), 3.0, dtype=od, device=DEV)
    moe.moe_mm_i8(xq, xs, wq, ws, o, row_token=t, out=keep)
    assert torch.equal(keep[:rows], got[:rows]) and (keep[rows:] == 3).all()


@pytest.mark.parametrize("R,N,K", [(1, 8, 16), (1, 4096, 7168), (3, 520, 1008), (17, 264, 272), (129, 136, 2048),
                                   (1030, 264, 144), (4099, 4096, 1024)])  # the last one in two launches
def test_mm_i8_dense(R, N, K):
    moe = M()
    g = gen(29)
    xq, xs = codes(g, R, K), torch.rand(R, device=DEV, generator=g) * 1e-2
    wq, ws = codes(g, N, K), torch.rand(N, device=DEV, generator=g) * 1e-3
    ref = (xq.double() @ wq.double().t()) * xs[:, None].double() * ws.double()
    near_i8(moe.moe_mm_i8(xq, xs, wq, ws, out_dtype=FP32), ref, "dense")
    t = torch.randint(-1, R + 1, (R,), device=DEV, generator=g).to(torch.int32)
    ok = (t >= 0) & (t < R)
    got = moe.moe_mm_i8(xq, xs, wq, ws, row_token=t, out_dtype=FP32)
    near_i8(got, ref[t.long().clamp(0, R - 1)] * ok[:, None], "gathered")


def test_mm_i8_largest_sums():
    """All codes -128 at the largest K: the sum 2^30 still fits an int32."""
    moe = M()
    K = 1 << 16
    xq = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((8, K), -128, dtype=torch.int8, device=DEV)
    y = moe.moe_mm_i8(xq, torch.ones(3, device=DEV), wq, torch.ones(8, device=DEV), out_dtype=FP32)
    assert (y == float(1 << 30)).all()


def ref_quant(v):
    """The quantisation rule in fp32 steps, each correctly rounded.  (A Python
    number over a tensor is no such step: PyTorch takes the reciprocal, then a product.)"""
    one, full = torch.ones(()), torch.full((), 127.0)
    m = full / v.abs().amax(1).clamp_min(2.0 ** -64)
    return torch.round(v * m[:, None]).to(torch.int8), one / m


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,K", [(1, 16), (5, 496), (3, 1024), (4, 1040), (2, 2064), (7, 4096), (3, 7168), (2, 16384),
                                 (2, 16400), (1, 40000), (1500, 512)])
def test_quant_i8(R, K, dtype):
    moe = M()
    g = gen(31)
    x = rand(g, R, K, dtype=dtype) * torch.logspace(-3, 2, R, device=DEV)[:, None].to(dtype)
    x[R // 2, K // 2] = 60000.0 if dtype == FP16 else 3e38  # one outlier
    if R > 2:
        x[1] = 0
    if R > 3:
        x[2] = 1e-7 if dtype == FP16 else 1e-38  # below the floor of the maximum (bf16)
    got, scale = moe.moe_quant_i8(x)
    want, ws = ref_quant(x.float().cpu())
    assert torch.equal(got.cpu(), want) and torch.equal(scale.cpu(), ws)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,K", [(1, 16), (37, 128), (5, 1536), (3, 2064), (2, 7168), (1, 16400)])
def test_quant_i8_swiglu(R, K, dtype):
    """v in fp32 is off by a few of its roundings (exponential 2, sum, quotient,
    product: under 16 2^-24), so v * m by 127 * 32 * 2^-24 < 3e-4 of a step."""
    moe = M()
    x = rand(gen(37), R, 2 * K, dtype=dtype) * 2
    got, scale = moe.moe_quant_i8(x, swiglu=True)
    v = x[:, :K].double() * torch.sigmoid(x[:, :K].double()) * x[:, K:].double()
    top = v.abs().amax(1)
    assert ((got.double() - v * 127 / top[:, None]).abs() <= 0.5 + 3e-4).all()
    assert ((scale.double() * 127 / top - 1).abs() <= 32 * 2.0 ** -24).all()


def test_quant_i8_rows_that_are_not_finite():
    moe = M()
    x = rand(gen(41), 6, 256)
    clean = moe.moe_quant_i8(x)
    x[1, 3], x[3, 255], x[4, 0] = float("nan"), float("inf"), float("-inf")
    q, s = moe.moe_quant_i8(x)
    bad = torch.tensor([False, True, False, True, True, False], device=DEV)
    assert torch.isnan(s[bad]).all() and not q[bad].any()
    assert torch.equal(q[~bad], clean[0][~bad]) and torch.equal(s[~bad], clean[1][~bad])
    # and their results are NaN, the others' are not (also where the product quantises by itself)
    for rows in (slice(0, 6), slice(1, 2), slice(2, 3), slice(4, 5)):
        y = moe.moe_linear_i8(x[rows].contiguous(), codes(gen(1), 64, 256), torch.ones(64, device=DEV))
        assert torch.isnan(y[bad[rows]]).all() and torch.isfinite(y[~bad[rows]]).all()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts,tail,N,K", [([1], 0, 64, 256), ([1], 0, 4096, 7168), ([1], 0, 24, 8192), ([1], 0, 72, 8208),
                                             ([0, 1, 0, 2], 1, 264, 144), ([0, 0, 1], 0, 264, 144), ([0, 0], 1, 40, 1024), ([0, 0], 3, 40, 1024),
                                             ([3, 0, 18, 1], 2, 264, 160), ([400, 0, 700], 9, 136, 272)])
def test_linear_i8_equals_its_two_steps(counts, tail, N, K, dtype, swiglu):
    moe = M()
    g = gen(43)
    o, R, E = offs(counts), sum(counts) + tail, len(counts)
    x = rand(g, R, 2 * K if swiglu else K, dtype=dtype)
    wq, ws = codes(g, E, N, K), torch.rand(E, N, device=DEV, generator=g) * 1e-3
    q, s = moe.moe_quant_i8(x, swiglu)
    want = moe.moe_mm_i8(q, s, wq, ws, o, out_dtype=dtype)
    assert torch.equal(moe.moe_linear_i8(x, wq, ws, o, swiglu=swiglu), want)
    work = torch.full((moe.moe_linear_i8_workspace_size(R, K),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((R, N), 2.0, dtype=FP32, device=DEV)
    moe.moe_linear_i8(x, wq, ws, o, swiglu=swiglu, out=out, work=work)
    rows = sum(counts)
    assert torch.equal(out[:rows], moe.moe_mm_i8(q, s, wq, ws, o, out_dtype=FP32)[:rows]) and (out[rows:] == 2).all()
    # gathered: each token twice
    t = torch.arange(R, device=DEV).flip(0).div(2, rounding_mode="floor").to(torch.int32)
    got = moe.moe_linear_i8(x, wq, ws, o, row_token=t, swiglu=swiglu)
    assert torch.equal(got, moe.moe_mm_i8(q, s, wq, ws, o, row_token=t, out_dtype=dtype))
    # some rows name no token
    for bad in (-1, R):
        t[::2] = bad
        got = moe.moe_linear_i8(x, wq, ws, o, row_token=t, swiglu=swiglu)
        assert torch.equal(got, moe.moe_mm_i8(q, s, wq, ws, o, row_token=t, out_dtype=dtype)) and not got[::2].any()
    # one row of many tokens
    t = torch.tensor([R - 1], dtype=torch.int32, device=DEV)
    one = offs([0] * (E - 1) + [1])
    got = moe.moe_linear_i8(x, wq, ws, one, row_token=t, swiglu=swiglu)
    assert torch.equal(got, moe.moe_mm_i8(q, s, wq, ws, one, row_token=t, out_dtype=dtype))
    if E == 1:  # dense
        assert torch.equal(moe.moe_linear_i8(x, wq[0], ws[0], swiglu=swiglu), want)


# ------------------------------------------------------------------ streams, graphs
def test_on_another_stream_and_replayed():
    """Captured calls take new values and new offsets at each replay, between eager work."""
    moe = M()
    g = gen(47)
    N, K, R = 136, 256, 200
    x, w, dy = rand(g, R, K), rand(g, 3, N, K), rand(g, R, N)
    wq, ws = codes(g, 3, N, K), torch.rand(3, N, device=DEV, generator=g) * 1e-3
    o = offs([20, 100, 80])
    work = torch.empty(moe.moe_linear_i8_workspace_size(R, K), dtype=torch.uint8, device=DEV)

    def run():
        return (moe.moe_grouped_mm(x, w, o), moe.moe_grouped_mm_dgrad(dy, w, o), moe.moe_grouped_mm_wgrad(dy, x, o),
                moe.moe_linear_i8(x, wq, ws, o, work=work))

    eager = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i, counts in enumerate(([20, 100, 80], [0, 200, 0], [1, 2, 150], [200, 0, 0])):
        x.copy_(rand(gen(100 + i), R, K))
        dy.copy_(rand(gen(200 + i), R, N))
        o.copy_(offs(counts))
        graph.replay()
        torch.cuda.synchronize()
        got = [h.clone() for h in held]
        assert all(torch.equal(a, b) for a, b in zip(got, run())), counts


def test_a_training_step_in_a_graph():
    """Forward and backward captured together, replayed with new values and other groups."""
    moe = M()
    g = gen(61)
    R, N, K = 150, 72, 128
    x, w = rand(g, R, K).requires_grad_(), rand(g, 3, N, K).requires_grad_()
    dy, o = rand(g, R, N), offs([50, 0, 90])

    def step():
        y = moe.moe_grouped_mm(x, w, o)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i, counts in enumerate(([50, 0, 90], [1, 149, 0], [0, 0, 3])):
        with torch.no_grad():
            x.copy_(rand(gen(300 + i), R, K))
        o.copy_(offs(counts))
        graph.replay()
        torch.cuda.synchronize()
        got = [h.clone() for h in held]
        xd, wd = x.detach(), w.detach()
        want = (moe.moe_grouped_mm(xd, wd, o), moe.moe_grouped_mm_dgrad(dy, wd, o), moe.moe_grouped_mm_wgrad(dy, xd, o))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), counts


# ------------------------------------------------------------------ together
def test_an_int8_expert_layer_from_the_parts():
    """Router, permute, int8 gate|up with rows gathered from the tokens, SwiGLU
    and quantisation in front of the down projection, combine: each part
    against 64 bits on what it was given, and the layer as a whole against the
    layer on unrounded intermediates.

    Bound of the whole, from what is rounded on the way: gate and up to bf16, d
    = 2^-8 of each; SwiGLU turns that into at most d (1 + |1 + g (1 - s(g))|)
    |h| (s the sigmoid: the relative slopes of its product and of silu); the
    codes add half a step of the largest |h|, and W2's rows sum these absolutely.
    The fp32 steps and the last bf16 rounding are 2^-8 of the result and
    1e-5 of its absolute sum."""
    moe = M()
    g = gen(53)
    T, H, I, E, k = 33, 256, 128, 8, 2
    x, gate = rand(g, T, H), rand(g, E, H, scale=0.05)
    cfg = moe.Cfg(T, H, I, E, k, 0, 32, 32)
    ids, tw = moe.moe_route(cfg, x, gate)
    _, o, eidx, rtok, _, _ = moe.moe_permute(cfg, x, ids)
    quant = lambda w: ((w / (w.abs().amax(2, keepdim=True) / 127)).round().to(torch.int8), w.abs().amax(2) / 127)
    w1, s1 = quant(torch.randn(E, 2 * I, H, device=DEV, generator=g) * 0.05)
    w2, s2 = quant(torch.randn(E, H, I, device=DEV, generator=g) * 0.05)
    gu = moe.moe_linear_i8(x, w1, s1, o, row_token=rtok)
    y = moe.moe_linear_i8(gu, w2, s2, o, swiglu=True, out_dtype=FP32)
    out = moe.moe_combine(cfg, y, eidx, o, tw)

    q, s = moe.moe_quant_i8(x)
    hq, hs = moe.moe_quant_i8(gu, swiglu=True)
    e_of = torch.repeat_interleave(torch.arange(E, device=DEV), (o[1:] - o[:-1]).long())
    t = rtok.long()
    d2 = w2.double() * s2.double()[:, :, None]
    # the codes' sums are exact, so scales come after them
    mm = lambda w, ws, c, cs: (w.double()[e_of] @ c.double()[:, :, None])[:, :, 0] * cs.double()[:, None] * ws.double()[e_of]
    v = mm(w1, s1, q[t], s[t])
    near_i8(gu, v, "gate and up")
    near_i8(y, mm(w2, s2, hq, hs), "down")
    gather = lambda r: (r[eidx.long()].view(T, k, H) * tw.double()[:, :, None]).sum(1)
    assert ((out.double() - gather(y.double())).abs() <= 2.0 ** -8 * 1.01 * gather(y.double()).abs()
            + 1e-5 * gather(y.double().abs())).all()

    sig = torch.sigmoid(v[:, :I])
    h = v[:, :I] * sig * v[:, I:]
    dh = 2.0 ** -8 * 1.02 * (1 + (1 + v[:, :I] * (1 - sig)).abs()) * h.abs()
    step = (h.abs() + dh).amax(1, keepdim=True) / 127
    ref = gather((d2[e_of] @ h[:, :, None])[:, :, 0])
    tol = gather((d2[e_of].abs() @ (dh + step / 2)[:, :, None])[:, :, 0])
    size = gather((d2[e_of].abs() @ h.abs()[:, :, None])[:, :, 0])
    assert ((out.double() - ref).abs() <= tol + 2.0 ** -8 * 1.01 * (ref.abs() + tol) + 1e-5 * size).all()


def test_a_16_bit_expert_layer_trains():
    """The experts in bf16 with their gradients, permuted by the framework's own
    routing: the weights' gradients against autograd in 64 bits.  Every bf16
    rounding (products' outputs, SwiGLU, gradients) is half a step, 2^-8, of a
    value; a handful of them in a row give under 5 % of the gradient's norm."""
    moe = M()
    g = gen(59)
    T, H, I, E, k = 64, 128, 128, 4, 2
    x = rand(g, T, H)
    cfg = moe.Cfg(T, H, I, E, k, 0, 32, 32)
    ids, tw = moe.moe_route(cfg, x, rand(g, E, H, scale=0.05))
    _, o, eidx, rtok, _, _ = moe.moe_permute(cfg, x, ids)
    w1, w2 = rand(g, E, 2 * I, H, scale=0.1).requires_grad_(), rand(g, E, H, I, scale=0.1).requires_grad_()

    def forward(x, w1, w2, mm):
        gu = mm(x[rtok.long()], w1)
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        y = mm(h, w2)
        return (y[eidx.long()].view(T, k, H) * tw[:, :, None].to(y.dtype)).sum(1)

    def mm64(a, w):
        return torch.cat([a[int(o[e]):int(o[e + 1])] @ w[e].t() for e in range(E)])

    dout = rand(g, T, H)
    got = torch.autograd.grad(forward(x, w1, w2, lambda a, w: moe.moe_grouped_mm(a, w, o)), (w1, w2), dout)
    d1, d2 = w1.detach().double().requires_grad_(), w2.detach().double().requires_grad_()
    want = torch.autograd.grad(forward(x.double(), d1, d2, mm64), (d1, d2), dout.double())
    for a, b in zip(got, want):
        assert (a.double() - b).norm() <= 0.05 * b.norm()
