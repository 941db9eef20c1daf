"""The row-major MXFP4 quantiser and products against plain 64-bit forms (needs
an MI355X).

Tolerances.  The quantiser of 16-bit values is exact: codes and scales are equal
to the rule's.  A product of two codes and their scales is exact in fp32, and K of
them summed in fp32 in any order are off by at most K 2^-23 sum |x w| (2^-23 rather
than 2^-24 per addition also covers an adder that truncates); the one rounding to
the output type adds eps / 2 of the value (fp16: or half its smallest subnormal).
With all scales 1 every partial sum is a multiple of 1/4 below 2^22, so the fp32
result is the exact one.
"""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LEVELS = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


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


def offs(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def rand_codes(g, *shape):
    return torch.randint(0, 256, shape, device=DEV, generator=g, dtype=torch.uint8)


def rand_scales(g, *shape, low=121, high=132):
    return torch.randint(low, high, shape, device=DEV, generator=g, dtype=torch.uint8)


def values(codes, scales):
    """What codes [..., K / 2] and scales [..., K / 32] stand for, in 64 bits."""
    level = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    return level[c] * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def rule(v):
    """Codes and scales of the rows of v (64 bits) by the definition."""
    R, K = v.shape
    b = v.view(R, -1, 32)
    top = b.abs().amax(2)
    fine = torch.isfinite(b).all(2)
    power = (torch.floor(torch.log2(top.clamp_min(2.0 ** -400))) - 2).clamp(-127, 127)
    u = b.abs() * torch.exp2(-power)[:, :, None]
    level = torch.tensor(LEVELS, dtype=torch.float64, device=v.device)
    mid = (level[1:] + level[:-1]) / 2
    lo, hi = torch.bucketize(u, mid), torch.bucketize(u, mid, right=True)
    code = torch.where(lo % 2 == 0, lo, hi) + 8 * torch.signbit(b)
    code = torch.where(fine[:, :, None], code, 0).view(R, K)
    scale = torch.where(fine, power + 127, 255.0)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scale.to(torch.uint8)


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_quant_every_value(dtype):
    """Every 16-bit pattern beside a block maximum of every exponent that keeps it in play."""
    moe = M()
    bits = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16).view(dtype)
    codes, scales = moe.moe_quant_mx4(bits.view(64, 1024))
    want, ws = rule(bits.double().view(64, 1024))
    assert torch.equal(codes, want) and torch.equal(scales, ws)
    spread = bits.view(32, 2048).t().contiguous()  # 32 exponents and signs to a block
    codes, scales = moe.moe_quant_mx4(spread)
    want, ws = rule(spread.double())
    assert torch.equal(codes, want) and torch.equal(scales, ws)
    finite = bits[torch.isfinite(bits)]
    finite = finite[torch.argsort(finite.abs().float(), stable=True)]
    pairs = torch.stack([finite[:-16], finite[16:]], 1)  # values beside slightly larger ones, at every scale
    rows = torch.zeros(pairs.shape[0], 32, dtype=dtype, device=DEV)
    rows[:, 5:7] = pairs
    codes, scales = moe.moe_quant_mx4(rows)
    want, ws = rule(rows.double())
    assert torch.equal(codes, want) and torch.equal(scales, ws)


@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (7, 4096), (61, 7168), (1003, 352), (4099, 2048), (3, 1 << 20)])
def test_quant(R, K):
    moe = M()
    note("test_quant", R, K)
    g = gen(R + K)
    for dtype in (BF16, FP16):
        x = torch.randn(R, K, device=DEV, generator=g).to(dtype)
        x[:, ::32] *= 4  # (ties and saturation: few mantissa bits)
        x[:, 1::3] = (x[:, 1::3] * 4).round() / 4
        codes, scales = moe.moe_quant_mx4(x)
        want, ws = rule(x.double())
        assert torch.equal(codes, want) and torch.equal(scales, ws)
        x[R // 2, K // 2] = float("nan")
        x[0, 0] = float("inf")
        codes, scales = moe.moe_quant_mx4(x)
        want, ws = rule(x.double())
        assert torch.equal(codes, want) and torch.equal(scales, ws) and scales[0, 0] == 255


def test_quant_swiglu():
    """h = silu(gate) * up in fp32 (a few roundings off): scales and codes of a value next to a border may be the neighbour's."""
    moe = M()
    for R, K in ((1, 32), (9, 96), (500, 2048)):
        g = gen(K)
        x = torch.randn(R, 2 * K, device=DEV, generator=g).to(BF16)
        codes, scales = moe.moe_quant_mx4(x, swiglu=True)
        gate, up = x.double().chunk(2, dim=1)
        h = gate * torch.sigmoid(gate) * up
        off = 8 * 2.0 ** -24  # exp, sum, quotient, product, and the exponent's error up to |gate| = 6
        top = h.view(R, -1, 32).abs().amax(2)
        low, high = (torch.floor(torch.log2(top * f)) - 2 + 127 for f in (1 - off, 1 + off))
        assert ((scales.double() == low) | (scales.double() == high)).all()
        unit = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
        u = h / unit
        half = torch.where(u.abs() < 2, 0.25, torch.where(u.abs() < 4, 0.5, 1.0))
        assert ((values(codes, scales) / unit - u.clamp(-6, 6)).abs() <= half * (1 + 1e-9) + off * u.abs()).all()
        want, ws = rule(h)
        assert (codes != want).double().mean() < 1e-3


def test_quant_into_the_callers_tensors():
    moe = M()
    g = gen(1)
    x = torch.randn(5, 256, device=DEV, generator=g).to(BF16)
    want = moe.moe_quant_mx4(x)
    codes, scales = torch.full((7, 128), 9, dtype=torch.uint8, device=DEV), torch.full((48,), 9, dtype=torch.uint8, device=DEV)
    got = moe.moe_quant_mx4(x, codes=codes[1:6], scales=scales[:40].view(5, 8))
    assert torch.equal(codes[1:6], want[0]) and torch.equal(scales[:40].view(5, 8), want[1])
    assert (codes[::6] == 9).all() and (scales[40:] == 9).all() and got[0].data_ptr() == codes[1:].data_ptr()
    e = moe.moe_quant_mx4(x[:0])
    assert e[0].shape == (0, 128) and e[1].shape == (0, 8)


# ------------------------------------------------------------------ products
def near(got, ref, mag, K, what):
    dt = got.dtype
    tol = (K + 8) * 2.0 ** -23 * mag + torch.finfo(dt).eps / 2 * 1.01 * ref.abs()
    tol = tol * 1.01 + (2.0 ** -25 if dt == FP16 else 1e-38)
    got = got.double()
    if dt == FP16:  # 65520, half a step past the largest value, and all above it round to infinity
        over = got.isinf() & (got.sign() == ref.sign()) & (ref.abs() + tol >= 65520)
        got = torch.where(over, ref, got)
    assert torch.isfinite(got).all(), what
    worst = ((got - ref).abs() / tol).max().item() if got.numel() else 0.0
    assert worst <= 1.0, (what, worst)


def reference(x, w, o):
    """x [R, K] and w [E, N, K] in 64 bits."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(o[e]), int(o[e + 1])
        y[a:b] = x[a:b] @ w[e].t()
        mag[a:b] = x[a:b].abs() @ w[e].abs().t()
    return y, mag


# (rows per group, rows behind the last group, N, K); K / 32 odd, a multiple of 2, of 4, of 16
SHAPES = {
    "one_row": ([1], 0, 8, 32),
    "one_row_of_many": ([0, 0, 1, 0], 0, 128, 256),
    "tiny_layer": ([5, 0, 7, 1, 3, 0, 13, 8], 0, 128, 256),
    "no_full_tile": ([3, 17, 64, 65], 0, 136, 224),
    "k_past_a_step": ([9, 33], 0, 264, 288),
    "odd_blocks": ([40, 3, 0, 21], 5, 72, 1056),
    "behind_the_last": ([4, 0, 70], 31, 72, 160),
    "only_behind": ([0, 0, 0], 77, 264, 64),
    "first_and_last_empty": ([0, 100, 129, 0], 3, 520, 992),
    "about_128_a_group": ([127, 128, 129, 0, 200], 0, 392, 320),
    "large_groups": ([511, 0, 700, 257], 65, 264, 448),
    "one_large_group": ([1025], 0, 1032, 512),
    "one_large_group_odd": ([1025], 0, 1000, 2016),
    "larger_groups": ([1300, 0, 2049, 7], 9, 776, 1184),
    "full_tiles": ([2048, 1024], 0, 2048, 2048),
    "skewed": ([900] + [0] * 30 + [1], 0, 256, 128),
    "many_groups": ([i % 5 for i in range(200)], 9, 64, 64),
    "most_groups": ([i % 3 for i in range(1024)], 5, 16, 32),
    "many_large_groups": ([257, 300, 0] * 45, 0, 72, 96),
    "long_k": ([2, 30], 0, 16, 16416),
    "long_k_large": ([600, 300], 0, 520, 8224),
    "decode_slice": ([1, 0, 2, 1, 0, 0, 3, 1], 0, 1536, 4096),
    "prefill_slice": ([300, 0, 511, 260, 1, 129, 64, 700], 0, 1536, 4096),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_products(name):
    moe = M()
    counts, tail, N, K = SHAPES[name]
    note("test_products", name)
    g = gen(N + K)
    o = offs(counts)
    R, E, rows = sum(counts) + tail, len(counts), sum(counts)
    xq, wq = rand_codes(g, R, K // 2), rand_codes(g, E, N, K // 2)
    xs, ws = rand_scales(g, R, K // 32), rand_scales(g, E, N, K // 32)
    y, mag = reference(values(xq, xs), values(wq, ws), o)
    for dt in (BF16, FP16, FP32):
        got = moe.moe_mm_mx4(xq, xs, wq, ws, o, out_dtype=dt)
        assert got.dtype == dt
        near(got, y, mag, K, dt)
        assert not got[rows:].any()
    # sums that fp32 holds exactly
    one = torch.full_like(xs, 127), torch.full_like(ws, 127)
    y, _ = reference(values(xq, one[0]), values(wq, one[1]), o)
    got = moe.moe_mm_mx4(xq, one[0], wq, one[1], o, out_dtype=FP32)
    assert torch.equal(got.double(), y)
    # rows of tokens, and a caller's tensor: rows of no group stay as they are
    T = max(1, R // 3)
    rt = torch.randint(0, T, (R,), device=DEV, generator=g, dtype=torch.int32)
    bad = torch.rand(R, device=DEV, generator=g) < 0.1
    rt[bad] = torch.where(torch.rand(int(bad.sum()), device=DEV, generator=g) < 0.5, -1, T).to(torch.int32)
    tq, ts = xq[:T].contiguous(), one[0][:T].contiguous()
    out = torch.full((R, N), 7.0, dtype=FP32, device=DEV)
    got = moe.moe_mm_mx4(tq, ts, wq, one[1], o, row_token=rt, out=out)
    x = values(tq, ts)[rt.clamp(0, T - 1).long()]
    x[bad] = 0
    y, _ = reference(x, values(wq, one[1]), o)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out[:rows].double(), y[:rows]) and (out[rows:] == 7).all()


@pytest.mark.parametrize("R,N,K", [(1, 8, 32), (1, 4096, 7168), (3, 136, 96), (17, 1000, 4064), (64, 4096, 4096),
                                   (200, 520, 1056), (300, 4096, 2048), (515, 1032, 480), (1030, 4096, 1024),
                                   (2051, 2056, 1120), (4099, 512, 256)])
def test_dense(R, N, K):
    moe = M()
    note("test_dense", R, N, K)
    g = gen(R + N + K)
    xq, wq = rand_codes(g, R, K // 2), rand_codes(g, N, K // 2)
    xs, ws = rand_scales(g, R, K // 32), rand_scales(g, N, K // 32)
    y, mag = reference(values(xq, xs), values(wq, ws)[None], [0, R])
    near(moe.moe_mm_mx4(xq, xs, wq, ws), y, mag, K, "dense")
    one = torch.full_like(xs, 127), torch.full_like(ws, 127)
    y = values(xq, one[0]) @ values(wq, one[1]).t()
    assert torch.equal(moe.moe_mm_mx4(xq, one[0], wq, one[1], out_dtype=FP32).double(), y)


@pytest.mark.parametrize("counts", [[3, 2], [300, 280]], ids=["few", "many"])
def test_scales_of_every_exponent(counts):
    """Scales from 2^-127 to 2^127, results up to infinity and down to fp32's subnormals; 255 is NaN, in its row alone."""
    moe = M()
    g = gen(9)
    R, N, K = sum(counts), 264, 544
    o = offs(counts)
    xq, wq = rand_codes(g, R, K // 2), rand_codes(g, 2, N, K // 2)
    xs, ws = rand_scales(g, R, 1, low=0, high=255).expand(R, K // 32).contiguous(), torch.full((2, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    ws[:, 5] = 7
    ws[:, 6] = 250
    got = moe.moe_mm_mx4(xq, xs, wq, ws, o, out_dtype=FP32)
    y, mag = reference(values(xq, xs), values(wq, ws), o)
    big, small = mag > 1e38, mag < 1e-30
    fine = ~big & ~small
    assert fine.double().mean() > 0.6
    tol = (K + 8) * 2.0 ** -23 * mag + 2.0 ** -23 * y.abs()
    assert ((got.double() - y).abs()[fine] <= tol[fine]).all()
    assert (got[small].abs() <= 1e-29).all()  # (sums of subnormals may be flushed)
    sure = big & (y.abs() > 3.5e38 * 1.01)
    assert (got[sure].isinf() | got[sure].isnan()).all()
    xs[1, 3] = 255
    ws[1, 9, 16] = 255
    clean = got
    got = moe.moe_mm_mx4(xq, xs, wq, ws, o, out_dtype=FP32)
    nan = torch.zeros(R, N, dtype=torch.bool, device=DEV)
    nan[1] = True
    nan[counts[0]:, 9] = True
    assert got[nan].isnan().all()
    assert torch.equal(got[~nan].view(torch.int32), clean[~nan].view(torch.int32))


def test_a_block_that_is_not_finite_stays_in_its_row():
    moe = M()
    g = gen(10)
    for R in (5, 700):
        x = torch.randn(R, 512, device=DEV, generator=g).to(BF16)
        w = torch.randn(264, 512, device=DEV, generator=g).to(BF16)
        wq, ws = moe.moe_quant_mx4(w)
        clean = moe.moe_linear_mx4(x, wq, ws)
        x[2, 100], x[4, 511] = float("inf"), float("nan")
        y = moe.moe_linear_mx4(x, wq, ws)
        assert y[2].isnan().all() and y[4].isnan().all()
        keep = [r for r in range(R) if r not in (2, 4)]
        assert torch.equal(y[keep], clean[keep])


LINEAR = [(1, 1, 0, 7168, 4096), (1, 1, 0, 96, 264), (2, 1, 0, 4096, 1024), (7, 1, 0, 224, 72), (16, 1, 0, 2048, 512),
          (17, 1, 0, 2080, 520), (600, 1, 0, 1056, 776), (1, 8, 64, 2048, 512), (1, 2, 8, 256, 128), (9, 4, 16, 544, 136),
          (61, 8, 64, 512, 264), (1, 8, 64, 16416, 16)]


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("T,topk,E,K,N", LINEAR)
def test_linear_is_the_two_calls(T, topk, E, K, N, swiglu):
    moe = M()
    note("test_linear", T, topk, E, K, N, swiglu)
    g = gen(T + K)
    for dtype in (BF16, FP16):
        wide = 2 * K if swiglu else K
        wq, ws = moe.moe_quant_mx4(torch.randn(max(1, E) * N, K, device=DEV, generator=g).to(dtype))
        x = torch.randn(T, wide, device=DEV, generator=g).to(dtype)
        if not E:
            want = moe.moe_mm_mx4(*moe.moe_quant_mx4(x, swiglu), wq, ws, out_dtype=dtype)
            got = moe.moe_linear_mx4(x, wq, ws, swiglu=swiglu)
            assert got.dtype == dtype and torch.equal(got, want)
            continue
        wq, ws = wq.view(E, N, -1), ws.view(E, N, -1)
        ids = torch.rand(T, E, device=DEV, generator=g).topk(topk, 1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        o = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=E).cumsum(0)]).to(torch.int32)
        rt = (order // topk).to(torch.int32)
        want = moe.moe_mm_mx4(*moe.moe_quant_mx4(x, swiglu), wq, ws, o, row_token=rt, out_dtype=FP32)
        work = torch.full((moe.moe_linear_mx4_workspace_size(T, K, T * topk),), 255, dtype=torch.uint8, device=DEV)
        got = moe.moe_linear_mx4(x, wq, ws, o, row_token=rt, swiglu=swiglu, out_dtype=FP32, work=work)
        assert torch.equal(got, want)
        rows = x[rt.long()].contiguous()
        assert torch.equal(moe.moe_linear_mx4(rows, wq, ws, o, swiglu=swiglu, out_dtype=FP32), want)


def test_offsets_of_a_longer_array_and_wrong_ones():
    """A run of a longer offset array; offsets that decrease or lie outside give wrong rows, never an access outside."""
    moe = M()
    g = gen(12)
    R, N, K, E = 90, 72, 160, 4
    xq, wq = rand_codes(g, R, K // 2), rand_codes(g, E, N, K // 2)
    xs, ws = torch.full((R, K // 32), 127, dtype=torch.uint8, device=DEV), torch.full((E, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    long = offs([13, 20, 0, 31, 9, 17])
    o = long[1:6]
    y = torch.zeros(R, N, dtype=torch.float64, device=DEV)
    for e in range(E):
        a, b = int(o[e]), int(o[e + 1])
        y[a:b] = values(xq[a:b], xs[a:b]) @ values(wq[e], ws[e]).t()
    assert torch.equal(moe.moe_mm_mx4(xq, xs, wq, ws, o, out_dtype=FP32).double(), y)
    for bad in ([0, 50, 20, 70, 90], [-5, 10, 300, 20, 1 << 30], [90, 80, 60, 10, 0]):
        got = moe.moe_mm_mx4(xq, xs, wq, ws, torch.tensor(bad, dtype=torch.int32, device=DEV), out_dtype=FP32)
        assert got.shape == (R, N)
    assert moe.moe_mm_mx4(xq[:0], xs[:0], wq, ws, o * 0).shape == (0, N)
    none = torch.zeros(R, dtype=torch.int32, device=DEV)
    assert not moe.moe_mm_mx4(xq[:0], xs[:0], wq, ws, o, row_token=none).any()  # no token: rows of zeros


@pytest.mark.parametrize("R,T,N,K", [(1, 5, 72, 96), (1, 5, 520, 8224), (40, 7, 136, 1056), (300, 1000, 264, 512), (1030, 64, 4096, 1024),
                                     (4099, 33, 512, 7168)])
def test_dense_rows_of_tokens(R, T, N, K):
    """One matrix, rows gathered from tokens, some of which name none: in one launch and in two."""
    moe = M()
    g = gen(R + T)
    wq, ws = moe.moe_quant_mx4(torch.randn(N, K, device=DEV, generator=g).to(BF16))
    x = torch.randn(T, K, device=DEV, generator=g).to(BF16)
    rt = torch.randint(0, T, (R,), device=DEV, generator=g, dtype=torch.int32)
    for bad in (False, True):
        if bad:
            rt[::3] = T
            rt[R // 2] = -7
        xq, xs = moe.moe_quant_mx4(x)
        got = moe.moe_mm_mx4(xq, xs, wq, ws, row_token=rt, out_dtype=FP32)
        live = (rt >= 0) & (rt < T)
        v = values(xq, xs)[rt.clamp(0, T - 1).long()] * live[:, None]
        y, mag = reference(v, values(wq, ws)[None], [0, R])
        near(got, y, mag, K, "gathered")
        assert not got[~live].any()
        assert torch.equal(moe.moe_linear_mx4(x, wq, ws, row_token=rt, out_dtype=FP32), got)


def test_two_calls_at_once():
    """Calls on two streams, each with scratch of its own, give what they give alone."""
    moe = M()
    g = gen(14)
    cases = []
    for R, N, K in ((600, 1032, 2048), (9, 4096, 1056)):
        wq, ws = moe.moe_quant_mx4(torch.randn(N, K, device=DEV, generator=g).to(BF16))
        x = torch.randn(R, K, device=DEV, generator=g).to(BF16)
        cases.append((x, wq, ws, moe.moe_linear_mx4(x, wq, ws)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for st, (x, wq, ws, want) in zip(streams, cases):
            with torch.cuda.stream(st):
                got.append((moe.moe_linear_mx4(x, wq, ws), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)


def test_streams_and_graph():
    moe = M()
    g = gen(13)
    st = torch.cuda.Stream()
    for R, N, K in ((1, 512, 2048), (300, 776, 1056), (1030, 1024, 512)):
        wq, ws = moe.moe_quant_mx4(torch.randn(N, K, device=DEV, generator=g).to(BF16))
        x = torch.randn(R, K, device=DEV, generator=g).to(BF16)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            got = moe.moe_linear_mx4(x * 1, wq, ws)
        st.synchronize()
        assert torch.equal(got, moe.moe_linear_mx4(x, wq, ws))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = moe.moe_linear_mx4(x, wq, ws)
        for k in range(3):
            x.copy_(torch.randn(R, K, device=DEV, generator=g))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(got, moe.moe_linear_mx4(x, wq, ws)), (R, k)
