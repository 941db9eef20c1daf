"""The 16-bit products where no rounding hides a lost row: operands are
multiples of 2^-4 up to 1/2, so a product is a multiple of 2^-8 up to 1/4, and a
sum of up to 2^17 of them is a multiple of 2^-8 up to 2^15: 23 bits, exact in
fp32 in any order.  fp32 results equal the 64-bit form, 16-bit ones its one
rounding (needs an MI355X)."""
import pytest
import torch

import bit_grouped_gemm_amd as moe
from test_gpu_mm import BF16, DEV, FP16, FP32, gen, note, offs, ref_fwd, ref_wgrad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load()
    yield


def small(g, *shape, dtype=BF16):
    return (torch.randint(-8, 9, shape, device=DEV, generator=g) / 16).to(dtype)


def rounded(ref, dtype):
    return ref.float().to(dtype)  # the first step is exact


def splits(R, N, K, E):
    """Workgroups that share a group's rows, by the scratch they need."""
    need = moe.moe_grouped_mm_wgrad_workspace_size(R, N, K, E)
    return need // (4 * E * N * K) if need else 1


# (rows per group, N, K, row splits): below, at and above the join's eight at a time, no multiple of it,
# the most there are; groups too short for their last splits; more steps than splits divide
SPLITS = [([700], 72, 136, 1), ([1613], 72, 136, 3), ([4100], 136, 72, 8), ([4500], 8, 8, 8), ([6700], 264, 72, 13),
          ([8193], 256, 256, 16), ([12345], 72, 264, 24), ([33001], 136, 264, 64), ([131000], 16, 24, 255),
          ([6000, 3, 0, 700], 72, 136, 3), ([1, 9000, 65, 64, 0], 136, 520, 3), ([0, 0, 20000], 40, 48, 13),
          ([20000, 0, 0], 520, 48, 13), ([600, 5000, 500], 264, 264, 4)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts,N,K,want", SPLITS, ids=str)
def test_wgrad_splits_lose_no_row(counts, N, K, want, dtype):
    R, E = sum(counts) + 50, len(counts)  # the last rows belong to no group
    note("test_wgrad_splits_lose_no_row", counts, N, K, dtype)
    assert splits(R, N, K, E) == want
    g = gen(3)
    dy, x, o = small(g, R, N, dtype=dtype), small(g, R, K, dtype=dtype), offs(counts)
    ref, _ = ref_wgrad(dy, x, o)
    for out in (FP32, dtype):
        assert torch.equal(moe.moe_grouped_mm_wgrad(dy, x, o, out_dtype=out), rounded(ref, out)), out


@pytest.mark.parametrize("E,N,K,rows", [(300, 264, 264, 9), (40, 776, 520, 20), (40, 776, 520, 200), (24, 520, 1000, 25),
                                        (9, 1032, 1032, 1300)], ids=str)
def test_wgrad_tiles_lose_no_row(E, N, K, rows):
    """Several tiles per workgroup (short groups), and one with three stages (long ones)."""
    counts = [0 if e % 5 == 2 else rows * (3 if e % 7 == 3 else 1) - e % 3 for e in range(E)]
    note("test_wgrad_tiles_lose_no_row", E, N, K, rows)
    g = gen(4)
    o, R = offs(counts), sum(counts)
    dy, x = small(g, R, N), small(g, R, K)
    ref, _ = ref_wgrad(dy, x, o)
    for out in (FP32, BF16):
        assert torch.equal(moe.moe_grouped_mm_wgrad(dy, x, o, out_dtype=out), rounded(ref, out)), out


@pytest.mark.parametrize("counts,N,K", [([1], 16, 8200), ([2, 30, 0, 5], 72, 4104), ([40, 0, 7, 130], 264, 2056),
                                        ([300, 700, 1, 400], 520, 1032), ([1500, 2000, 0, 900], 1032, 776),
                                        ([3000, 1100, 5000], 264, 2120), ([5], 8200, 16), ([900, 0, 3], 2056, 264)], ids=str)
def test_products_lose_no_column(counts, N, K):
    """Forward and dx over long reductions of odd lengths, in every tile height."""
    note("test_products_lose_no_column", counts, N, K)
    g = gen(5)
    o, R, E = offs(counts), sum(counts), len(counts)
    x, dy, w = small(g, R, K), small(g, R, N), small(g, E, N, K)
    y, _ = ref_fwd(x, w, o)
    dx, _ = ref_fwd(dy, w.transpose(1, 2).contiguous(), o)
    for out in (FP32, BF16):
        assert torch.equal(moe.moe_grouped_mm(x, w, o, out_dtype=out), rounded(y, out)), out
        assert torch.equal(moe.moe_grouped_mm_dgrad(dy, w, o, out_dtype=out), rounded(dx, out)), out


# ------------------------------------------------------------------ what is not finite stays in its group
@pytest.mark.parametrize("out", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,N,K,want", [([9 + e % 4 if e % 6 else 0 for e in range(300)], 264, 264, 1),  # in turns
                                             ([200 + e % 5 for e in range(40)], 776, 520, 1),          # three stages
                                             ([3000, 0, 2500, 3100, 2000], 72, 136, 4)], ids=["turns", "stages", "splits"])
def test_wgrad_of_groups_between_groups_that_are_not_finite(counts, N, K, want, out):
    """Every other group, and the rows of no group before and behind, hold NaN and
    infinities: the other groups' gradients keep their bits."""
    E, head, tail = len(counts), 37, 70
    R = head + sum(counts) + tail
    note("test_wgrad_of_groups_between", E, N, K, R, out)
    assert splits(R, N, K, E) == want
    g = gen(6)
    o = offs(counts) + head
    dy, x = small(g, R, N), small(g, R, K)
    ref, _ = ref_wgrad(dy, x, o)
    bounds = o.tolist()
    bad = [(0, head), (R - tail, R)] + [(bounds[e], bounds[e + 1]) for e in range(0, E, 2)]
    for t, which in ((dy, float("nan")), (x, float("inf"))):
        for a, b in bad:
            t[a:b] = which
            t[a:b:3] = float("-inf")
    dw = torch.full((E, N, K), 3.0, dtype=out, device=DEV)
    moe.moe_grouped_mm_wgrad(dy, x, o.to(torch.int32), out=dw)
    for e in range(E):
        if e % 2 or not counts[e]:
            assert torch.equal(dw[e], rounded(ref[e], out)), e
        else:
            assert not torch.isfinite(dw[e]).any(), e
    # a run of the groups: the rows of the others belong to none
    part = moe.moe_grouped_mm_wgrad(dy, x, o.to(torch.int32)[1:E], out_dtype=out)
    assert splits(R, N, K, E - 2) >= 1
    for e in range(1, E - 1, 2):
        assert torch.equal(part[e - 1], rounded(ref[e], out)), e


@pytest.mark.parametrize("counts,N,K", [([9 + e % 4 if e % 6 else 0 for e in range(300)], 264, 264),
                                        ([200 + e % 5 for e in range(40)], 776, 520), ([300, 700, 1, 400], 520, 1032),
                                        ([1, 0, 2, 1, 3], 264, 2056)], ids=["short", "middle", "long", "few"])
def test_rows_of_groups_between_groups_that_are_not_finite(counts, N, K):
    E, head, tail = len(counts), 21, 40
    R = head + sum(counts) + tail
    note("test_rows_of_groups_between", E, N, K, R)
    g = gen(7)
    o = (offs(counts) + head).to(torch.int32)
    x, dy, w = small(g, R, K), small(g, R, N), small(g, E, N, K)
    y, _ = ref_fwd(x, w, o)
    dx, _ = ref_fwd(dy, w.transpose(1, 2).contiguous(), o)
    bounds = o.tolist()
    for a, b in [(0, head), (R - tail, R)] + [(bounds[e], bounds[e + 1]) for e in range(0, E, 2)]:
        x[a:b], dy[a:b] = float("nan"), float("inf")
    w[::2] = float("nan")
    got, gdx = moe.moe_grouped_mm(x, w, o, out_dtype=FP32), moe.moe_grouped_mm_dgrad(dy, w, o, out_dtype=FP32)
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if e % 2:
            assert torch.equal(got[a:b], y[a:b].float()) and torch.equal(gdx[a:b], dx[a:b].float()), e
        else:
            assert torch.isnan(got[a:b]).all() and torch.isnan(gdx[a:b]).all(), e
    for t in (got, gdx):
        assert not t[:head].any() and not t[R - tail:].any()
