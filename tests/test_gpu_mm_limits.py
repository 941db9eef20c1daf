"""The row-major products and the int8 quantiser at the borders of what a launch
and an int32 hold (needs an MI355X).

A launch counts its work items in 32 bits, and a larger count wraps without an
error: so every row of these results is looked at, and what is left unwritten
shows.  Rows that are not under test are zeros, and outputs start as something else."""
import pytest
import torch

import bit_grouped_gemm_amd as moe
from test_gpu_mm import BF16, DEV, FP16, FP32, codes, gen, near, near_i8, note, rand, ref_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load()
    yield


@pytest.fixture(autouse=True)
def _memory():
    """These tests take tens of GB each."""
    yield
    torch.cuda.empty_cache()


def all_equal(t, value):
    """Every element of t, in pieces (a comparison of the whole would need as much again)."""
    return all(bool((part == value).all()) for part in t.reshape(-1).split(1 << 30))


# ------------------------------------------------------------------ more rows than a launch has work items
# four rows per workgroup up to K = 1024, one beyond: 2^26 and 2^24 rows are 2^32 work items
@pytest.mark.parametrize("R,K,swiglu", [((1 << 26) - 4, 16, False), ((1 << 26) - 3, 16, False), (1 << 26, 16, False),
                                        ((1 << 26) + 4, 16, True), (3 * (1 << 26) + 1, 16, False),
                                        ((1 << 24) - 1, 1040, False), (1 << 24, 1040, False), ((1 << 24) + 8, 1040, True)])
def test_quant_i8_rows_past_a_launch(R, K, swiglu):
    note("test_quant_i8_rows_past_a_launch", R, K, swiglu)
    g = gen(3)
    width = 2 * K if swiglu else K
    x = torch.zeros(R, width, dtype=BF16, device=DEV)
    # around the end of a first launch, and the last rows
    border = min((1 << 26 if K <= 1024 else 1 << 24) - 4, R - 16)
    for a in (border - 8, R - 16):
        x[a:a + 16] = rand(g, 16, width)
    q = torch.full((R, K), 99, dtype=torch.int8, device=DEV)
    s = torch.full((R,), -1.0, device=DEV)
    moe.moe_quant_i8(x, swiglu, codes=q, scales=s)
    zero = moe.moe_quant_i8(torch.zeros(1, width, dtype=BF16, device=DEV), swiglu)[1]
    for a in (border - 8, R - 16):
        want = moe.moe_quant_i8(x[a:a + 16].contiguous(), swiglu)
        assert torch.equal(q[a:a + 16], want[0]) and torch.equal(s[a:a + 16], want[1])
    for a in (border - 8, R - 16):
        q[a:a + 16], s[a:a + 16] = 0, zero
    assert all_equal(q, 0) and all_equal(s, zero)


def test_linear_i8_rows_past_a_launch():
    g = gen(4)
    R, K, N = (1 << 26) + 5, 16, 8
    note("test_linear_i8_rows_past_a_launch", R)
    x = torch.zeros(R, K, dtype=FP16, device=DEV)
    x[-16:] = rand(g, 16, K, dtype=FP16)
    wq, ws = codes(g, N, K), torch.rand(N, device=DEV, generator=g) * 1e-2
    y = torch.full((R, N), 7.0, dtype=FP32, device=DEV)
    moe.moe_linear_i8(x, wq, ws, out=y)
    assert torch.equal(y[-16:], moe.moe_linear_i8(x[-16:].contiguous(), wq, ws, out_dtype=FP32))
    assert all_equal(y[:-16], 0)


# 2^30 rows of 8 outputs are 2^24 of the 64-row tiles that narrow products take, 2^32 work items
@pytest.mark.parametrize("R", [(1 << 30) - 192, (1 << 30) + (1 << 20) + 37])
@pytest.mark.parametrize("name", ["moe_grouped_mm", "moe_grouped_mm_dgrad"])
def test_products_of_more_tiles_than_a_launch(name, R):
    note("test_products_of_more_tiles_than_a_launch", name, R)
    g = gen(5)
    x = torch.zeros(R, 8, dtype=BF16, device=DEV)
    some = (0, R // 2, R - 300)  # rows that are looked at; all others are zeros
    for a in some:
        x[a:a + 300] = rand(g, 300, 8)
    w = rand(g, 2, 8, 8)
    o = torch.tensor([0, R - 200, R], dtype=torch.int32, device=DEV)
    y = torch.full((R, 8), 7.0, dtype=BF16, device=DEV)
    getattr(moe, name)(x, w, o, out=y)
    wf = w if name == "moe_grouped_mm" else w.transpose(1, 2).contiguous()
    for a in some:
        ref, mag = ref_fwd(x[a:a + 300], wf, torch.tensor([0, 100 if a == some[2] else 300, 300]))
        near(y[a:a + 300], ref, mag, 8, "y")
        y[a:a + 300] = 0
    assert all_equal(y, 0)


@pytest.mark.parametrize("R", [(1 << 30) - 64, (1 << 30) + 64])
def test_mm_i8_of_more_tiles_than_a_launch(R):
    note("test_mm_i8_of_more_tiles_than_a_launch", R)
    g = gen(6)
    xq = torch.zeros(R, 16, dtype=torch.int8, device=DEV)
    some = (0, R // 2, R - 300)
    for a in some:
        xq[a:a + 300] = codes(g, 300, 16)
    xs = torch.full((R,), 0.5, device=DEV)
    wq, ws = codes(g, 8, 16), torch.rand(8, device=DEV, generator=g)
    y = torch.full((R, 8), 7.0, dtype=BF16, device=DEV)
    moe.moe_mm_i8(xq, xs, wq, ws, out=y)
    for a in some:
        near_i8(y[a:a + 300], xq[a:a + 300].double() @ wq.double().t() * 0.5 * ws.double(), "y")
        y[a:a + 300] = 0
    assert all_equal(y, 0)


# ------------------------------------------------------------------ wrong offsets
@pytest.mark.parametrize("E,R", [(1024, 360_000_000), (1024, 300_000_000), (2, 1000)])
def test_offsets_that_name_rows_many_times_stay_inside_the_tensors(E, R):
    """Offsets 0, R, 0, R, ...: every second group claims all rows, and of 1024
    groups their 64-row tiles pass an int32.  What comes out is not defined, but
    nothing outside the result is written."""
    note("test_offsets_that_name_rows_many_times", E, R)
    g = gen(7)
    margin = 1 << 20
    x, w = torch.zeros(R, 8, dtype=BF16, device=DEV), rand(g, E, 8, 8)
    o = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32, device=DEV)
    flat = torch.full((R + 2 * margin, 8), 5.0, dtype=BF16, device=DEV)
    moe.moe_grouped_mm(x, w, o, out=flat[margin:margin + R])
    torch.cuda.synchronize()
    assert all_equal(flat[:margin], 5) and all_equal(flat[margin + R:], 5)
    # zeros times weights, or left alone
    assert all(bool(((p == 0) | (p == 5)).all()) for p in flat.reshape(-1).split(1 << 30))


# ------------------------------------------------------------------ one launch or two
@pytest.mark.parametrize("K", [1024, 7168])
@pytest.mark.parametrize("R", [256, 257, 300, 523, 1030, 2051, 4096, 4101])
def test_mm_i8_dense_in_one_launch_or_two(R, K):
    """Row counts on both sides of the rule that gives the last rows a launch of
    their own: each row comes out as it does alone, whichever it is."""
    g = gen(8)
    N = 4096
    xq, xs = codes(g, R, K), torch.rand(R, device=DEV, generator=g) * 1e-2
    wq, ws = codes(g, N, K), torch.rand(N, device=DEV, generator=g) * 1e-3
    y = torch.full((R, N), 7.0, dtype=FP32, device=DEV)
    moe.moe_mm_i8(xq, xs, wq, ws, out=y)
    t = torch.arange(R, dtype=torch.int32, device=DEV)
    assert torch.equal(y, moe.moe_mm_i8(xq, xs, wq, ws, row_token=t, out_dtype=FP32))
    for a in (0, R // 256 * 256 - 5, R - 5):  # the first rows, those around the border, the last
        a = max(a, 0)
        some = xq[a:a + 10].contiguous(), xs[a:a + 10].clone()
        assert torch.equal(y[a:a + 10], moe.moe_mm_i8(*some, wq, ws, out_dtype=FP32))
    near_i8(y, xq.double() @ wq.double().t() * xs.double()[:, None] * ws.double(), "y")
