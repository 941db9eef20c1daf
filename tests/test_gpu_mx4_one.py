"""moe_linear_mx4 of one row through wide projections, which it quantises inside the
product (needs an MI355X).

Tolerance: the codes are the quantiser's, products of codes and scales exact in
fp32, and K of them summed in fp32 in any order off by at most K 2^-23 sum |x w|; the
rounding to the output type adds eps / 2 of the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LEVELS = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def values(codes, scales):
    table = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=DEV)
    both = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    power = torch.tensor([2.0 ** (e - 127) for e in range(255)] + [float("nan")], dtype=torch.float64, device=DEV)
    return (both.unflatten(-1, (scales.shape[-1], 32)) * power[scales.int()][..., None]).flatten(-2)


@pytest.mark.parametrize("K,N", [(4096, 28672), (4096, 57344), (4064, 151936), (8192, 12288), (96, 40008), (8224, 28680)])
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
def test_one_row_of_a_wide_projection(K, N, swiglu):
    import bit_grouped_gemm_amd as moe
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("test_one_row_of_a_wide_projection", K, N, swiglu, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(K + N)
    wq = torch.randint(0, 256, (N, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    ws = torch.randint(119, 126, (N, K // 32), device=DEV, generator=g, dtype=torch.uint8)
    for dtype in (BF16, FP16):
        x = torch.randn(1, 2 * K if swiglu else K, device=DEV, generator=g).to(dtype)
        v = values(*moe.moe_quant_mx4(x, swiglu))[0]
        y, mag = torch.empty(N, dtype=torch.float64, device=DEV), torch.empty(N, dtype=torch.float64, device=DEV)
        for a in range(0, N, 8192):
            w = values(wq[a:a + 8192], ws[a:a + 8192])
            y[a:a + 8192], mag[a:a + 8192] = w @ v, w.abs() @ v.abs()
        for out in (dtype, FP32):
            tol = K * 2.0 ** -23 * mag + torch.finfo(out).eps / 2 * 1.01 * y.abs() + (2.0 ** -25 if out == FP16 else 1e-38)
            for got in (moe.moe_linear_mx4(x, wq, ws, swiglu=swiglu, out_dtype=out),
                        moe.moe_mm_mx4(*moe.moe_quant_mx4(x, swiglu), wq, ws, out_dtype=out)):
                assert got.shape == (1, N) and torch.isfinite(got).all()
                assert ((got[0].double() - y).abs() <= tol).all(), (K, N, out)


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
def test_one_row_that_is_not_finite_or_of_no_group(swiglu):
    """A block with an infinity or NaN makes the row NaN; a row of no group, or one that names no token, is zeros
    whatever x holds, and stays as it is in a caller's tensor."""
    import bit_grouped_gemm_amd as moe
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    K, N, E = 1344, 264, 3
    wq = torch.randint(0, 256, (E, N, K // 2), device=DEV, generator=g, dtype=torch.uint8)
    ws = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    x = torch.randn(1, 2 * K if swiglu else K, device=DEV, generator=g).to(BF16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    clean = moe.moe_linear_mx4(x, wq[1].contiguous(), ws[1].contiguous(), swiglu=swiglu, out_dtype=FP32)
    assert torch.isfinite(clean).all() and clean.any()
    assert torch.equal(moe.moe_linear_mx4(x, wq, ws, i32(0, 0, 1, 1), swiglu=swiglu, out_dtype=FP32), clean)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[0, 700] = bad
        assert moe.moe_linear_mx4(y, wq[1].contiguous(), ws[1].contiguous(), swiglu=swiglu).isnan().all()
        for o in ((0, 0, 0, 0), (1, 1, 1, 1)):
            assert not moe.moe_linear_mx4(y, wq, ws, i32(*o), swiglu=swiglu).any()
            out = torch.full((1, N), 7.0, dtype=BF16, device=DEV)
            moe.moe_linear_mx4(y, wq, ws, i32(*o), swiglu=swiglu, out=out)
            assert (out == 7).all()
        for t in (-1, 1, 1 << 30):
            assert not moe.moe_linear_mx4(y, wq, ws, i32(0, 0, 1, 1), row_token=i32(t), swiglu=swiglu).any()
        both = torch.cat([y, x])
        assert torch.equal(moe.moe_linear_mx4(both, wq, ws, i32(0, 0, 1, 1), row_token=i32(1), swiglu=swiglu, out_dtype=FP32), clean)
    wn = ws[1].clone()
    wn[9, 3] = 255
    y = moe.moe_linear_mx4(x, wq[1].contiguous(), wn, swiglu=swiglu, out_dtype=FP32)
    assert y[0, 9].isnan() and torch.equal(y[0, :9], clean[0, :9]) and torch.equal(y[0, 10:], clean[0, 10:])
