"""The RMS norm, its quantised forms and its gradients against plain 64-bit
forms (needs an MI355X).

Tolerances.  A lane adds at most 32 squares in a row and the rest meet in
trees, so the sum of squares is off by at most 64 roundings (2^-24 each) of
itself and rstd by half of that plus the roundings of mean, eps, square root and
quotient; n = s * rstd and y = n * weight round twice more: kN = 48 roundings of
y in all.  The one rounding to 16 bits adds eps / 2 of the value (fp16: or half
its smallest subnormal).  In the backward pass mean(g n) has the error of a sum
of terms |g n|, and dx that of its three terms; 128 roundings of the sum of
their magnitudes cover it.  dweight adds a chain of R / 256 rows at most, and
fewer than 64 partial sums on top.
"""
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
kN = 48 * 2.0 ** -24
EPS = 1e-6


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


def rounding(ref, dtype):
    return torch.finfo(dtype).eps / 2 * 1.01 * ref.abs() + (2.0 ** -25 if dtype == FP16 else 1e-38)


def within(got, ref, tol, what):
    assert torch.isfinite(got.double()).all(), what
    worst = ((got.double() - ref).abs() / tol).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, (what, worst)


def same(a, b):
    """Equal bits, NaN's among them."""
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.dtype == b.dtype and torch.equal(a.view(kind), b.view(kind))


def reference(x, w, res, eps=EPS):
    """s (in x's type), n and y in 64 bits."""
    s = x if res is None else (x.float() + res.float()).to(x.dtype)
    v = s.double()
    rstd = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    return s, v * rstd, v * rstd * w.double(), rstd


# (R, K): one row; around a wave's, a workgroup's and the largest rows; rows that end inside a chunk of lanes
SHAPES = [(1, 8), (3, 64), (5, 512), (2, 520), (7, 1024), (1, 1032), (9, 2048), (4, 2056), (33, 4096), (3, 4104),
          (1, 7168), (6, 8192), (5, 8200), (2, 16384), (1003, 264), (777, 1536)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,K", SHAPES)
def test_norm(R, K, dtype):
    moe = M()
    note("test_norm", R, K, dtype)
    g = gen(R * 31 + K)
    x, res = rand(g, R, K, dtype=dtype, scale=0.7), rand(g, R, K, dtype=dtype, scale=3.0)
    for w in (rand(g, K, dtype=dtype), rand(g, K, dtype=FP32)):
        for r in (None, res):
            s, _, y, _ = reference(x, w, r)
            got = moe.moe_rms_norm(x, w, r, eps=EPS)
            if r is not None:
                got, total = got
                assert total.dtype == dtype and torch.equal(total, s)
            assert got.dtype == dtype
            within(got, y, kN * y.abs() + rounding(y, dtype) * (1 + 2.0 ** -10), "y")


@pytest.mark.parametrize("eps", [1e-30, 1e-12, 1e-3, 1.0])
def test_eps_and_zero_rows(eps):
    moe = M()
    g = gen(3)
    x = rand(g, 6, 256, scale=1e-3)
    x[2] = 0
    x[4] = 1e-12
    w = rand(g, 256, dtype=FP32)
    got = moe.moe_rms_norm(x, w, eps=eps)
    y = reference(x, w, None, torch.tensor(eps, dtype=FP32).double().item())[2]
    assert not got[2].any()
    within(got, y, kN * y.abs() + rounding(y, BF16) * 1.001, "y")


def test_largest_and_smallest_values():
    """Rows whose squares pass fp32's range, and fp16's largest values."""
    moe = M()
    g = gen(4)
    w = rand(g, 4096, dtype=FP32)
    x = rand(g, 5, 4096, scale=1e30)
    x[1, 7] = 3.38e38
    x[2] = 3.38e38
    x[3] = rand(g, 4096)
    x[3, 9] = -3e38
    y = reference(x, w, None)[2]
    got = moe.moe_rms_norm(x, w, eps=EPS)
    # (values under 2^-126 * 2^80 of the scaled row lose bits: none of these moves y by a rounding)
    within(got, y, kN * y.abs() + rounding(y, BF16) * 1.001 + 1e-30, "bf16")
    x = rand(g, 3, 4096, dtype=FP16)
    x[0] = 65504
    x[1, ::2] = -65504
    x[2] = 6e-8
    y = reference(x, w, None)[2]
    within(moe.moe_rms_norm(x, w, eps=EPS), y, kN * y.abs() + rounding(y, FP16) * 1.001, "fp16")


def test_not_finite():
    """An infinity or NaN stays in its row, and comes out as the formula has it."""
    moe = M()
    g = gen(5)
    inf, nan = float("inf"), float("nan")
    for K in (256, 4096):
        x, w = rand(g, 5, K), torch.ones(K, dtype=BF16, device=DEV)
        clean = moe.moe_rms_norm(x, w)
        x[1, 3], x[3, K - 1], x[3, 0] = inf, nan, -inf
        y = moe.moe_rms_norm(x, w)
        assert torch.equal(y[::2], clean[::2])
        assert y[1, 3].isnan() and not y[1, :3].any() and not y[1, 4:].any()
        assert y[3].isnan().all()
        for fmt in (moe.QFMT_E4M3, moe.QFMT_I8, moe.QFMT_MXFP4):
            codes, scales, _, _ = moe.moe_rms_norm_quant(x, w, fmt=fmt)
            x2 = x.clone()
            x2[1], x2[3] = 1, 1
            want, wants, _, _ = moe.moe_rms_norm_quant(x2, w, fmt=fmt)
            assert torch.equal(codes[::2], want[::2]) and torch.equal(scales[::2], wants[::2])
            # (a finite group of row 1 holds the formula's zeros, with their values' signs)
            sign = {moe.QFMT_E4M3: 0x80, moe.QFMT_I8: 0, moe.QFMT_MXFP4: 0x88}[fmt]
            assert not (codes[1] & ~sign).any() and not codes[3].any()
            assert not codes[1, :16].any()
            bad = (scales == 255) if fmt == moe.QFMT_MXFP4 else scales.isnan()
            if fmt == moe.QFMT_I8:
                assert bad.tolist() == [False, True, False, True, False]
            else:
                assert bad[1, 0] and not bad[1, 1:].any() and bad[3].all() and not bad[::2].any()


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def mx4_values(codes, scales):
    level = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    return level[c], torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


Q_SHAPES = [(1, 128), (3, 512), (5, 640), (2, 1024), (9, 1152), (4, 2048), (61, 4096), (3, 4224), (2, 7168), (1, 8192),
            (3, 8320), (2, 16384), (1003, 256)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,K", Q_SHAPES)
def test_quant(R, K, dtype):
    moe = M()
    note("test_quant", R, K, dtype)
    g = gen(R + K)
    x, res = rand(g, R, K, dtype=dtype), rand(g, R, K, dtype=dtype, scale=2.0)
    x[:, : K // 2] *= torch.exp(torch.randn(R, 1, device=DEV, generator=g) * 3).to(dtype)  # blocks of different size
    w = rand(g, K, dtype=FP32)
    w[K // 4: K // 4 + 32] = 0  # a whole block of zeros
    for r in (None, res):
        s, _, y, _ = reference(x, w, r)
        y16 = moe.moe_rms_norm(x, w, r, eps=EPS)
        y16 = y16 if r is None else y16[0]
        # the rows' sizes take a few fp16 values past the type's range: those rows are test_not_finite's
        fine = torch.isfinite(s).all(1)
        assert fine.sum() > 0.9 * R
        y = y[fine]
        wrong, n = kN * y.abs(), y.shape[0]

        def call(**kw):
            codes, scales, got, total = moe.moe_rms_norm_quant(x, w, r, eps=EPS, want_y=True, **kw)
            assert same(got, y16)
            assert total is None if r is None else same(total, s)
            alone = moe.moe_rms_norm_quant(x, w, r, eps=EPS, **kw)
            assert torch.equal(alone[0], codes) and same(alone[1], scales) and alone[2] is None
            return codes[fine], scales[fine]

        for group in (32, 128):
            codes, scales = call(fmt=moe.QFMT_E4M3, group=group)
            top = y.view(n, -1, group).abs().amax(2).clamp_min(2.0 ** -64)
            within(scales, top / 448, (kN + 4 * 2.0 ** -24) * top / 448, "e4m3 scales")
            v = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(group, 1)
            step = scales.double().repeat_interleave(group, 1) * 2.0 ** -10
            within(v, y, torch.maximum(2.0 ** -4 * y.abs(), step) * 1.001 + wrong, "e4m3")
        codes, scales = call(fmt=moe.QFMT_I8)
        top = y.abs().amax(1).clamp_min(2.0 ** -64)
        within(scales, top / 127, (kN + 4 * 2.0 ** -24) * top / 127, "int8 scales")
        within(codes.double() * scales.double()[:, None], y, scales.double()[:, None] * 0.501 + wrong, "int8")
        codes, scales = call(fmt=moe.QFMT_MXFP4)
        # the exponent is that of the greatest |y|, which a power of two may lie next to
        top = y.view(n, -1, 32).abs().amax(2)
        low, high = ((torch.floor(torch.log2((top * f).clamp_min(2.0 ** -200))) - 2).clamp(-127, 127) + 127
                     for f in (1 - kN, 1 + kN))
        assert ((scales.double() == low) | (scales.double() == high)).all()
        v, unit = mx4_values(codes, scales)
        u = y / unit
        half = torch.where(u.abs() < 2, 0.25, torch.where(u.abs() < 4, 0.5, 1.0))
        within(v, u.clamp(-6, 6), half * 1.001 + kN * u.abs(), "e2m1")


def test_mxfp4_rounding():
    """Every e2m1 boundary and its neighbours, over scales: exact values through the
    norm with rstd 1 (a row of mean square 1 - eps, weights that place the value)."""
    moe = M()
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    vals = [0.0, 6.0, 7.0, 7.75]
    for m in mids:
        vals += [m, m - 2.0 ** -12, m + 2.0 ** -12]
    vals = [s * v for v in vals for s in (1, -1)]
    K = 32 * len(vals)
    w = torch.zeros(K, dtype=FP32, device=DEV)
    want = torch.zeros(K, dtype=torch.float64, device=DEV)
    ties = {0.25: 0, 0.75: 1, 1.25: 1, 1.75: 2, 2.5: 2, 3.5: 4, 5.0: 4}
    for i, v in enumerate(vals):
        w[32 * i] = 4.0       # the block's greatest: X = 1
        w[32 * i + 1] = v
        want[32 * i] = 4
        a = abs(v)
        near = min(E2M1, key=lambda c: (abs(c - a), 0))
        want[32 * i + 1] = math.copysign(ties.get(a, 6 if a > 5 else near), v)
    x = torch.ones(1, K, dtype=BF16, device=DEV)
    # mean(s^2) + eps = 1 + 1e-30 rounds to 1: y is the weight itself
    codes, scales, _, _ = moe.moe_rms_norm_quant(x, w, eps=1e-30, fmt=moe.QFMT_MXFP4)
    v, unit = mx4_values(codes, scales)
    assert (unit == 1).all()
    assert torch.equal(v[0], want)
    # the same with the block's scale at every exponent that fp32 weights reach
    for e in list(range(-126, 125, 7)) + [124, 125]:
        codes2, scales2, _, _ = moe.moe_rms_norm_quant(x, w * 2.0 ** e, eps=1e-30,
                                                       fmt=moe.QFMT_MXFP4)
        if e >= -125 + 2:
            assert torch.equal(codes2, codes) and (scales2 == 127 + e).all(), e


# ------------------------------------------------------------------ gradients
def reference_grads(s, w, dy, ds, eps=EPS):
    """dx, dw in 64 bits, and the magnitudes their errors count from."""
    v, w, dy = s.double(), w.double(), dy.double()
    rstd = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    n, g = v * rstd, dy * w
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    mag = rstd * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if ds is not None:
        dx, mag = dx + ds.double(), mag + ds.double().abs()
    return dx, mag, (dy * n).sum(0), (dy * n).abs().sum(0)


def check_grads(moe, s, w, dy, ds, dx, dw):
    R = s.shape[0]
    want, mag, wdw, mdw = reference_grads(s, w, dy, ds)
    within(dx, want, 128 * 2.0 ** -24 * mag + rounding(want, dx.dtype) * 1.001, "dx")
    tol = (R / 256 + 64 + 64) * 2.0 ** -24 * mdw
    within(dw, wdw, tol + (rounding(wdw, dw.dtype) if dw.dtype != FP32 else 2.0 ** -24 * wdw.abs()) + 1e-30, "dw")


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,K", SHAPES + [(513, 4096), (2050, 1024), (5000, 72), (600, 8192)])
def test_gradients(R, K, dtype):
    moe = M()
    note("test_gradients", R, K, dtype)
    g = gen(R + 7 * K)
    x, res = rand(g, R, K, dtype=dtype), rand(g, R, K, dtype=dtype)
    dy, ds = rand(g, R, K, dtype=dtype, scale=0.1), rand(g, R, K, dtype=dtype, scale=0.1)
    for wt in (dtype, FP32):
        w = rand(g, K, dtype=wt).requires_grad_()
        a, b = x.clone().requires_grad_(), res.clone().requires_grad_()
        y, s = moe.moe_rms_norm(a, w, b, eps=EPS)
        da, db, dw = torch.autograd.grad((y, s), (a, b, w), (dy, ds))
        assert torch.equal(da, db) and dw.dtype == wt
        check_grads(moe, s.detach(), w.detach(), dy, ds, da, dw)
        y = moe.moe_rms_norm(a, w, eps=EPS)
        da, dw = torch.autograd.grad(y, (a, w), dy)
        check_grads(moe, x, w.detach(), dy, None, da, dw)
        # the same bits again, and from the entry point that autograd stands on
        y = moe.moe_rms_norm(a, w, eps=EPS)
        da2, dw2 = torch.autograd.grad(y, (a, w), dy)
        assert torch.equal(da, da2) and torch.equal(dw, dw2)


def test_gradient_against_differences():
    """The formula the kernels are held to, against central differences of the norm in 64 bits,
    and the kernels' own gradients against both."""
    moe = M()
    g = gen(11)
    R, K = 5, 136
    x, w = rand(g, R, K), rand(g, K, dtype=FP32)
    dy = rand(g, R, K)

    def loss(v, weight):
        return (v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * weight * dy.double()).sum()

    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(moe.moe_rms_norm(a, b, eps=EPS), (a, b), dy)
    want, mag, wdw, mdw = reference_grads(x, w, dy, None)
    h = 2.0 ** -17
    for k in range(0, K, 9):
        for r in range(R):
            d = torch.zeros(R, K, dtype=torch.float64, device=DEV)
            d[r, k] = h
            diff = (loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())) / (2 * h)
            # the difference's own error: h^2 / 6 of a third derivative of a few units, 2^-52 of the loss over h
            assert abs(diff - want[r, k]) <= 1e-8 * (1 + mag[r, k])
            assert abs(diff - dx[r, k].double()) <= 1e-8 * (1 + mag[r, k]) + 128 * 2.0 ** -24 * mag[r, k] + 2.0 ** -8 * abs(diff)
        d = torch.zeros(K, dtype=torch.float64, device=DEV)
        d[k] = h
        diff = (loss(x.double(), w.double() + d) - loss(x.double(), w.double() - d)) / (2 * h)
        assert abs(diff - dw[k].double()) <= 1e-8 * (1 + mdw[k]) + 200 * 2.0 ** -24 * mdw[k]


def test_gradients_wanted_one_by_one():
    moe = M()
    g = gen(12)
    x, res, w, dy, ds = (rand(g, 9, 512) for _ in range(5))
    w = w[0].contiguous()

    def grads(names, outs):
        t = {"x": x.clone(), "res": res.clone(), "w": w.clone()}
        for n in names:
            t[n].requires_grad_()
        y, s = moe.moe_rms_norm(t["x"], t["w"], t["res"], eps=EPS)
        pick = {"y": (y, dy), "s": (s, ds)}
        got = torch.autograd.grad([pick[o][0] for o in outs], [t[n] for n in names], [pick[o][1] for o in outs],
                                  allow_unused=True)
        return dict(zip(names, got))

    every = grads(("x", "res", "w"), ("y", "s"))
    for n in ("x", "res", "w"):
        assert torch.equal(grads((n,), ("y", "s"))[n], every[n])
    only_s = grads(("x", "res"), ("s",))
    assert torch.equal(only_s["x"], ds) and torch.equal(only_s["res"], ds)
    assert grads(("w", "x"), ("s",))["w"] is None
    only_y = grads(("x", "w"), ("y",))
    s = (x.float() + res.float()).to(BF16)
    check_grads(moe, s, w, dy, None, only_y["x"], only_y["w"])
    # frozen weight and no gradient at all
    assert not moe.moe_rms_norm(x, w).requires_grad
    with torch.no_grad():
        assert not moe.moe_rms_norm(x.clone().requires_grad_(), w).requires_grad


def test_expanded_and_unaligned_gradients():
    moe = M()
    g = gen(13)
    x, w = rand(g, 6, 264).requires_grad_(), rand(g, 264).requires_grad_()
    moe.moe_rms_norm(x, w).sum().backward()  # dy is one value, expanded
    one = torch.ones(6, 264, dtype=BF16, device=DEV)
    check_grads(moe, x.detach(), w.detach(), one, None, x.grad, w.grad)
    dy = rand(g, 6 * 264 + 1)[1:].view(6, 264)  # two bytes off
    dx, dw = torch.autograd.grad(moe.moe_rms_norm(x, w), (x, w), dy)
    check_grads(moe, x.detach(), w.detach(), dy, None, dx, dw)
    dy = rand(g, 264, 6).t()
    dx, dw = torch.autograd.grad(moe.moe_rms_norm(x, w), (x, w), dy)
    check_grads(moe, x.detach(), w.detach(), dy.contiguous(), None, dx, dw)
    y = moe.moe_rms_norm(x, w)
    with pytest.raises(RuntimeError):  # once differentiable
        (d,) = torch.autograd.grad(y, x, dy, create_graph=True)
        d.sum().backward()


def test_a_shared_weight_and_a_saved_sum_that_changes():
    moe = M()
    g = gen(14)
    x, w = rand(g, 8, 512).requires_grad_(), rand(g, 512).requires_grad_()
    y1, s = moe.moe_rms_norm(x, w, x)  # x is both summands, the weight is used twice
    y2 = moe.moe_rms_norm(s, w)
    dy = rand(g, 8, 512)
    dx, dw = torch.autograd.grad((y1, y2), (x, w), (dy, dy))
    both = 2 * reference_grads(s.detach(), w.detach(), dy, None)[2]
    within(dw, both, 2.0 ** -7 * both.abs() + 1e-2, "dw")  # two rounded gradients, and their rounded sum
    y, s = moe.moe_rms_norm(x, w, x)
    with torch.no_grad():
        s.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()


def test_entry_point_and_no_rows():
    moe = M()
    g = gen(15)
    x, w, dy, ds = rand(g, 70, 1032), rand(g, 1032, dtype=FP32), rand(g, 70, 1032), rand(g, 70, 1032)
    rstd = 1 / torch.sqrt(x.float().square().mean(1) + EPS)
    work = torch.empty(moe.moe_rms_norm_backward_workspace_size(70, 1032), dtype=torch.uint8, device=DEV).fill_(255)
    dx, dw = moe.moe_rms_norm_backward(dy, ds, x, rstd, w, EPS, work=work)
    check_grads(moe, x, w, dy, ds, dx, dw)
    e = x[:0]
    for r in (None, e):
        y = moe.moe_rms_norm(e, w, r)
        assert (y if r is None else y[0]).shape == (0, 1032)
    dx, dw = moe.moe_rms_norm_backward(e, None, e, rstd[:0], w, EPS)
    assert dx.shape == (0, 1032) and not dw.any()
    codes, scales, _, _ = moe.moe_rms_norm_quant(e[:, :1024].contiguous(), w[:1024].contiguous(), fmt=moe.QFMT_MXFP4)
    assert codes.shape == (0, 512) and scales.shape == (0, 32)
    xg, wg = e.clone().requires_grad_(), w.clone().requires_grad_()
    moe.moe_rms_norm(xg, wg).sum().backward()
    assert xg.grad.shape == (0, 1032) and not wg.grad.any()


def test_outputs_of_the_caller():
    moe = M()
    g = gen(16)
    x, res, w = rand(g, 21, 2056), rand(g, 21, 2056), rand(g, 2056)
    y, s = moe.moe_rms_norm(x, w, res)
    room = rand(g, 23, 2056)
    edge = room[::22].clone()
    out = room[1:22]
    r2 = res.clone()
    got, total = moe.moe_rms_norm(x, w, r2, out=out, sum_out=r2)  # the residual stream in place
    assert got.data_ptr() == out.data_ptr() and total.data_ptr() == r2.data_ptr()
    assert torch.equal(out, y) and torch.equal(r2, s) and torch.equal(room[::22], edge)
    x2 = x.clone()
    got, total = moe.moe_rms_norm(x2, w, res, sum_out=x2)
    assert torch.equal(got, y) and torch.equal(x2, s)
    x2 = x.clone()
    assert torch.equal(moe.moe_rms_norm(x2, w, out=x2), moe.moe_rms_norm(x, w))
    r2, xq = res[:, :2048].contiguous(), x[:, :2048].contiguous()
    want = moe.moe_rms_norm_quant(xq, w[:2048].contiguous(), r2)
    got = moe.moe_rms_norm_quant(xq, w[:2048].contiguous(), r2, sum_out=r2)
    assert got[3].data_ptr() == r2.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip((want[0], want[1], want[3]), (got[0], got[1], got[3])))
    with pytest.raises(ValueError, match="same tensor"):
        moe.moe_rms_norm(x, w, res, out=out, sum_out=out)
    with pytest.raises(ValueError):
        moe.moe_rms_norm(x, w, res, out=out.t())
    with pytest.raises(ValueError):
        moe.moe_rms_norm(x, w, res, sum_out=out.half())


def test_streams_and_graph():
    moe = M()
    g = gen(17)
    x, res, w, dy = rand(g, 300, 4096), rand(g, 300, 4096), rand(g, 4096), rand(g, 300, 4096)
    want = moe.moe_rms_norm(x, w, res)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        xs = x * 1
        got = moe.moe_rms_norm(xs, w, res)
        q = moe.moe_rms_norm_quant(xs, w, res)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b, c = x.clone().requires_grad_(), w.clone().requires_grad_(), res.clone().requires_grad_()

    def step():
        y, s = moe.moe_rms_norm(a, b, c)
        grads = torch.autograd.grad((y, s), (a, b, c), (dy, dy))
        return (y.detach(), s.detach(), *grads)  # (kept results hold no graph of the leaves)

    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        out = step()
    for k in range(4):
        with torch.no_grad():
            a.copy_(rand(g, 300, 4096))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, eager)), k


@pytest.mark.parametrize("residual", [False, True])
def test_a_graph_of_the_gradients_is_refused(residual):
    """Gradients asked for with create_graph are the same, and have none of their own."""
    moe = M()
    g = gen(5)
    x, w, dy = rand(g, 9, 264), rand(g, 264), rand(g, 9, 264)
    leaves = [t.requires_grad_() for t in ([x, w, rand(g, 9, 264)] if residual else [x, w])]

    def grads(dy, **kw):
        out = moe.moe_rms_norm(*leaves)
        return torch.autograd.grad(out[0] if residual else out, leaves, dy, **kw)

    plain, graph = grads(dy), grads(dy, create_graph=True)
    for a, b in zip(plain, graph):
        assert torch.equal(a, b) and not a.requires_grad
    with pytest.raises(RuntimeError):
        graph[0].sum().backward()
    graph = grads(dy.requires_grad_(), create_graph=True)  # linear in dy, which autograd must not pass over
    assert all(torch.equal(a, b) for a, b in zip(plain, graph))
    with pytest.raises(RuntimeError, match="once_differentiable"):
        graph[0].sum().backward()
