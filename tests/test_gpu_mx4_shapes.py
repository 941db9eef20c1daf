"""The MXFP4 product in every kernel and tile that it is ever made with, dense and
grouped, and in the two launches of a dense product with a few rows too many
(needs an MI355X; that each case takes the shape it is named by, and that all
shapes are here, is checked in test_mx4_shapes_cpu.py).

Tolerances: a product of two codes and their scales is exact in fp32, and K of
them summed in fp32 in any order are off by at most K 2^-23 sum |x w|; the one
rounding to the output type adds eps / 2 of the value.  With all scales 1 every
partial sum is a multiple of 1/4 below 2^22, so the fp32 result is the exact one.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LEVELS = [0, 0.5, 1, 1.5, 2, 3, 4, 6]

# (shape, rows, N, K, groups; 0: dense).  K ends inside a K step and a group of four, N inside a tile.
CASES = [
    ("few_16x16", 1, 24, 1344, 0), ("few_16x32", 1, 8200, 1344, 0), ("few_16x64", 4029, 40, 1472, 0),
    ("few_32x16", 4125, 40, 1344, 0), ("few_32x32", 8195, 24, 1344, 0), ("few_32x64", 6277, 40, 1408, 0),
    ("few_64x16", 15736, 16, 1504, 0), ("few_64x32", 4001, 72, 1472, 0), ("few_64x64", 8212, 40, 1344, 0),
    ("rows_16x64", 6214, 72, 1504, 0), ("rows_16x128", 8005, 72, 2528, 0), ("rows_16x256", 262, 3808, 3008, 0),
    ("rows_32x128", 8603, 72, 1344, 0), ("rows_32x256", 8010, 136, 2400, 0), ("rows_64x128", 16359, 40, 2464, 0),
    ("big_128x256", 18240, 136, 1376, 0), ("big_256x256", 16423, 264, 1344, 0),
    ("few_16x16", 1, 24, 1344, 2), ("few_16x32", 2, 4152, 1376, 2), ("few_16x64", 2, 8072, 1472, 2),
    ("few_32x16", 3267, 40, 1344, 107), ("few_32x32", 2910, 40, 1376, 161), ("few_32x64", 2862, 40, 1440, 196),
    ("few_64x16", 14924, 16, 1536, 43), ("few_64x32", 9249, 24, 1504, 162), ("few_64x64", 2824, 72, 1344, 101),
    ("rows_16x64", 545, 72, 1376, 182), ("rows_16x128", 8086, 72, 2016, 12), ("rows_16x256", 158, 928, 3040, 69),
    ("rows_32x128", 7222, 72, 1344, 126), ("rows_32x256", 4902, 144, 2400, 196), ("rows_64x128", 15548, 40, 2528, 25),
    ("big_128x256", 17403, 72, 1728, 192), ("big_256x256", 9863, 280, 1440, 125),
    # a decode batch's down projection; large tiles of few groups, a row tile more than the last column block has
    ("rows_16x128", 488, 7168, 2048, 64), ("big_256x256", 4100, 4104, 1056, 3),
    # the large tiles' rows, then the rest
    ("big_256x256+rows_16x64", 4099, 4096, 1056, 0), ("big_256x256+few_32x32", 4160, 4096, 7168, 0),
    ("big_256x256+few_16x16", 16411, 792, 1440, 0),
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def values(codes, scales):
    """The fp64 values of packed codes and e8m0 scales."""
    table = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=DEV)
    both = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    power = torch.tensor([2.0 ** (e - 127) for e in range(256)], dtype=torch.float64, device=DEV)
    return (both.unflatten(-1, (scales.shape[-1], 32)) * power[scales.int()][..., None]).flatten(-2)


def split(R, E, g):
    """Offsets of E ragged groups of R rows, some empty, with rows before the first and behind the last."""
    if R < 8:
        return torch.tensor([0] * E + [R], dtype=torch.int32, device=DEV)
    cut = torch.rand(E + 1, device=DEV, generator=g).sort().values
    cut = 0.01 + 0.98 * cut
    cut[0], cut[-1] = 0.01, 0.99
    if E > 2:
        cut[E // 2] = cut[E // 2 + 1]
    return (cut * R).to(torch.int32)


@pytest.mark.parametrize("shape,R,N,K,E", CASES, ids=[f"{s}-{E}x{R}x{N}x{K}" for s, R, N, K, E in CASES])
def test_shapes(shape, R, N, K, E):
    import bit_grouped_gemm_amd as moe
    print("test_shapes", shape, R, N, K, E, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(R + N + K + E)
    codes = lambda *s: torch.randint(0, 256, s, device=DEV, generator=g, dtype=torch.uint8)
    scales = lambda *s: torch.randint(121, 132, s, device=DEV, generator=g, dtype=torch.uint8)
    lead = (E, N) if E else (N,)
    xq, xs, wq, ws = codes(R, K // 2), scales(R, K // 32), codes(*lead, K // 2), scales(*lead, K // 32)
    o = split(R, E, g) if E else None
    bounds = o.tolist() if E else [0, R]
    mine = torch.zeros(R, dtype=torch.bool, device=DEV)
    mine[bounds[0]:bounds[-1]] = True

    def reference(x, w):
        y, mag = (torch.zeros(R, N, dtype=torch.float64, device=DEV) for _ in range(2))
        w = w if E else w[None]
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            y[a:b] = x[a:b] @ w[e].t()
            mag[a:b] = x[a:b].abs() @ w[e].abs().t()
        return y, mag

    y, mag = reference(values(xq, xs), values(wq, ws))
    for dt in (BF16, FP16, FP32):
        got = moe.moe_mm_mx4(xq, xs, wq, ws, o, out_dtype=dt)
        assert got.dtype == dt and got.shape == (R, N)
        # (past fp16's range a result is infinite, as it must be)
        tol = K * 2.0 ** -23 * mag + torch.finfo(dt).eps / 2 * 1.01 * y.abs() + (2.0 ** -25 if dt == FP16 else 1e-38)
        far = ~torch.isfinite(got)
        assert not far.any() or dt == FP16 and (y.abs() + tol >= 65520)[far].all()
        assert ((got.double() - y).abs() <= tol)[~far].all()
        assert not got[~mine].any()
    del mag
    # sums that fp32 holds exactly, of rows of tokens some of which name none, into the middle of a caller's tensor
    one, wone = torch.full_like(xs, 127), torch.full_like(ws, 127)
    T = max(1, R // 3)
    rt = torch.randint(0, T, (R,), device=DEV, generator=g, dtype=torch.int32)
    if R > 2:
        rt[1::7], rt[2::11] = -1, T
    live = (rt >= 0) & (rt < T)
    tq, ts = xq[:T].contiguous(), one[:T].contiguous()
    x = values(tq, ts)[rt.clamp(0, T - 1).long()] * live[:, None]
    y, _ = reference(x, values(wq, wone))
    room = torch.full((R + 4, N), 7.0, dtype=FP32, device=DEV)
    moe.moe_mm_mx4(tq, ts, wq, wone, o, row_token=rt, out=room[2:-2])
    assert torch.equal(room[2:-2][mine].double(), y[mine])
    assert (room[2:-2][~mine] == 7).all() and (room[:2] == 7).all() and (room[-2:] == 7).all()
    # the same as new rows, and rows by themselves, in 32 and in 16 bits
    new = moe.moe_mm_mx4(tq, ts, wq, wone, o, row_token=rt, out_dtype=FP32)
    assert torch.equal(new[mine], room[2:-2][mine]) and not new[~mine].any()
    y, _ = reference(values(xq, one), values(wq, wone))
    assert torch.equal(moe.moe_mm_mx4(xq, one, wq, wone, o, out_dtype=FP32).double(), y)
    assert torch.equal(moe.moe_mm_mx4(xq, one, wq, wone, o), y.float().to(BF16))  # (y is exact in fp32)
