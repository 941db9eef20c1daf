"""Sizes whose rows take more than one launch, or whose bytes or chunks pass 32 bits:
the norm, the MXFP4 quantiser and the MXFP4 products (needs an MI355X).  Rows do not
depend on each other, so those at the ends and around a launch's last row are held to
the same rows in a small call, bit for bit; products to exact sums (all scales 1:
every partial sum is a multiple of 1/4 below 2^22)."""
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
    yield
    torch.cuda.empty_cache()


def room_for(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free GPU memory")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def fill(t, g, scale=1.0):
    """Random values, of a block of rows again and again with another size."""
    block = torch.randn((1 << 20) // t.shape[1] + 1, t.shape[1], device=DEV, generator=g) * scale
    for i, part in enumerate(t.split(block.shape[0])):
        part.copy_(block[:part.shape[0]] * (0.5 + (i * 37 % 64) / 64))
    return t


LAUNCH = ((1 << 32) - 1) // 256 * 4  # rows of up to 1024 values that one launch has


@pytest.mark.parametrize("form", ["plain", "e4m3", "i8", "mxfp4"])
def test_norm_of_more_rows_than_a_launch_has(form):
    import bit_grouped_gemm_amd as moe
    K = {"plain": 8, "e4m3": 32, "i8": 16, "mxfp4": 32}[form]
    R = LAUNCH + 1003
    room_for(40)
    print("test_norm_of_more_rows_than_a_launch_has", form, R, K, flush=True)
    g = gen(K)
    x = fill(torch.empty(R, K, dtype=BF16, device=DEV), g)
    res = fill(torch.empty(R, K, dtype=BF16, device=DEV), g, 2.0)
    w = torch.randn(K, device=DEV, generator=g)
    parts = [slice(0, 70), slice(LAUNCH - 5, LAUNCH + 9), slice(R - 3, R), slice(R // 2, R // 2 + 99)]
    if form == "plain":
        got = [moe.moe_rms_norm(x, w, res)]
        small = [[moe.moe_rms_norm(x[p].clone(), w, res[p].clone())] for p in parts]
        # with rstd beside it, for the gradients of all rows
        a = x.requires_grad_()
        y, s = moe.moe_rms_norm(a, w, res)
        assert torch.equal(y, got[0][0]) and torch.equal(s, got[0][1])
        (dx,) = torch.autograd.grad(y, a, res)
        for p in parts:
            b = x[p].detach().clone().requires_grad_()
            (d,) = torch.autograd.grad(moe.moe_rms_norm(b, w, res[p].clone())[0], b, res[p].clone())
            assert torch.equal(d, dx[p]), p
    else:
        kw = {"e4m3": dict(fmt=moe.QFMT_E4M3, group=32), "i8": dict(fmt=moe.QFMT_I8), "mxfp4": dict(fmt=moe.QFMT_MXFP4)}[form]
        got = [moe.moe_rms_norm_quant(x, w, res, want_y=True, **kw)]
        small = [[moe.moe_rms_norm_quant(x[p].clone(), w, res[p].clone(), want_y=True, **kw)] for p in parts]
    for p, want in zip(parts, small):
        for a, b in zip(got[0], want[0]):
            assert torch.equal(a[p], b), (form, p)
            assert b.float().abs().sum() > 0


@pytest.mark.parametrize("K", [1 << 20, (1 << 20) - 32])
def test_swiglu_quantiser_past_32_bits_of_chunks(K):
    """More than 2^32 chunks of eight values, where a row's number takes a 64-bit division."""
    import bit_grouped_gemm_amd as moe
    R = 32771
    assert R * K // 8 > 1 << 32
    room_for(180)
    print("test_swiglu_quantiser_past_32_bits_of_chunks", R, K, flush=True)
    g = gen(1)
    x = torch.zeros(R, 2 * K, dtype=BF16, device=DEV)
    rows = [0, 1, 16385, R - 3, R - 2, R - 1]
    for r in rows:
        x[r] = torch.randn(2 * K, device=DEV, generator=g)
    codes, scales = moe.moe_quant_mx4(x, swiglu=True)
    for r in rows:
        c, s = moe.moe_quant_mx4(x[r:r + 1].clone(), swiglu=True)
        assert torch.equal(codes[r:r + 1], c) and torch.equal(scales[r:r + 1], s) and c.any(), r
    for r in (2, 16384, 16386, R - 4):  # zeros stay zeros
        assert not codes[r].any() and not scales[r].any(), r


def values(codes):
    table = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=DEV)
    return torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)


def random_codes(g, *shape):
    """Random bytes, of a block again and again (rolled by another number of bytes each time)."""
    t = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = t.view(-1)
    block = torch.randint(0, 256, (1 << 26,), device=DEV, generator=g, dtype=torch.uint8)
    for i, part in enumerate(flat.split(block.numel())):
        part.copy_(block.roll(i * 4099)[:part.numel()])
    return t


# (rows, N, K, groups; 0: dense): weights, results, rows past 2^32 bytes; the last is made in two launches
FAR = [(5, 65536, 65536, 3), (300, 65536, 65536, 3), (700, 65536, 65536, 3), (3, 262144, 65536, 0), (70001, 16392, 64, 0),
       (70001, 16392, 64, 5), (140001, 72, 65568, 0), (140001, 72, 65568, 3), (131073, 8200, 2080, 0)]


@pytest.mark.parametrize("R,N,K,E", FAR)
def test_products_past_32_bits(R, N, K, E):
    import bit_grouped_gemm_amd as moe
    room_for(60)
    print("test_products_past_32_bits", R, N, K, E, flush=True)
    g = gen(R)
    lead = (E, N) if E else (N,)
    ones = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=DEV)
    xq, wq = random_codes(g, R, K // 2), random_codes(g, *lead, K // 2)
    xs, ws = ones(R, K // 32), ones(*lead, K // 32)
    assert max(xq.numel(), wq.numel(), R * N * 4) > 1 << 32
    o = torch.tensor([R * e // max(E, 1) for e in range(max(E, 1) + 1)], dtype=torch.int32, device=DEV)
    got = moe.moe_mm_mx4(xq, xs, wq, ws, o if E else None, out_dtype=FP32)
    rows = torch.tensor(sorted({0, 1, R // 2, R - 2, R - 1} | {R * e // max(E, 1) for e in range(E)}), device=DEV)
    cols = torch.tensor(sorted({0, 7, N // 2, N // 2 + 1, N - 8, N - 1}), device=DEV)

    def want(x):
        y = torch.zeros(len(rows), len(cols), dtype=torch.float64, device=DEV)
        for i, r in enumerate(rows.tolist()):
            e = int((o[1:] <= r).sum()) if E else 0
            w = wq[e] if E else wq
            y[i] = values(w[cols]) @ values(x[r])
        return y

    assert torch.equal(got[rows][:, cols].double(), want(xq))
    assert torch.equal(moe.moe_mm_mx4(xq, xs, wq, ws, o if E else None)[rows][:, cols], want(xq).float().to(BF16))
