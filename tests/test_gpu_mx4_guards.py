"""MXFP4 products beside memory that is not theirs: rows and groups of NaN scales in
front of and behind the operands, a pattern around the result.  Offsets that
decrease or lie outside give wrong rows, but nothing outside is read into a result
or written (needs an MI355X; the kernels clamp every offset to the rows there are)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
FP32 = torch.float32
GUARD = 16  # rows or groups, so that what follows stays aligned


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def between(t, fill):
    """t between GUARD rows or groups of `fill` on either side."""
    room = torch.full((t.shape[0] + 2 * GUARD, *t.shape[1:]), fill, dtype=t.dtype, device=DEV)
    room[GUARD:-GUARD] = t
    return room, room[GUARD:-GUARD]


def wrong_offsets(R, E, g):
    up = torch.linspace(0, R, E + 1, device=DEV).to(torch.int32)
    yield "right", up
    yield "down", up.flip(0).contiguous()
    yield "zigzag", torch.where(torch.arange(E + 1, device=DEV) % 2 == 0, up, R - up).to(torch.int32)
    yield "outside", torch.randint(-2 * R, 3 * R, (E + 1,), device=DEV, generator=g, dtype=torch.int32)
    yield "far", torch.tensor([-(1 << 31), (1 << 31) - 1], dtype=torch.int32, device=DEV).repeat(E)[:E + 1].contiguous()
    yield "all_of_it", torch.tensor([0, 1 << 30], dtype=torch.int32, device=DEV).repeat(E)[:E + 1].contiguous()


# the same sizes as in the tests of every shape: large tiles of few and of many groups, the others
@pytest.mark.parametrize("R,N,K,E", [(90, 72, 160, 4), (4100, 4104, 1056, 3), (9863, 280, 1440, 125), (17403, 72, 1728, 192),
                                     (2824, 72, 1344, 101), (545, 72, 1376, 182), (2, 8072, 1472, 2)])
def test_wrong_offsets(R, N, K, E):
    import bit_grouped_gemm_amd as moe
    g = torch.Generator(device=DEV)
    g.manual_seed(R + N)
    codes = lambda *s: torch.randint(0, 256, s, device=DEV, generator=g, dtype=torch.uint8)
    ones = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=DEV)
    T = max(1, R // 2)
    held = [between(t, v) for t, v in ((codes(R, K // 2), 0x77), (ones(R, K // 32), 255), (codes(E, N, K // 2), 0x77),
                                       (ones(E, N, K // 32), 255))]
    xq, xs, wq, ws = (h[1] for h in held)
    before = [h[0].clone() for h in held]
    tokens = torch.randint(-3, T + 3, (R + 2 * GUARD,), device=DEV, generator=g, dtype=torch.int32)
    tokens[:GUARD] = tokens[-GUARD:] = 1 << 30
    rt = tokens[GUARD:-GUARD]
    tq, ts = between(xq[:T], 0x77)[1], between(xs[:T], 255)[1]
    for name, o in wrong_offsets(R, E, g):
        print("test_wrong_offsets", R, N, K, E, name, flush=True)
        for a, b, t in ((xq, xs, None), (tq, ts, rt)):
            room, out = between(torch.full((R, N), 3e38, dtype=FP32, device=DEV), -3e38)
            moe.moe_mm_mx4(a, b, wq, ws, o, row_token=t, out=out)
            assert (room[:GUARD] == -3e38).all() and (room[-GUARD:] == -3e38).all()
            assert torch.isfinite(out).all()
            new = moe.moe_mm_mx4(a, b, wq, ws, o, row_token=t, out_dtype=FP32)
            assert new.shape == (R, N)
            if name == "right":
                assert torch.equal(new, out)
        x = torch.randn(R, K, device=DEV, generator=g).to(torch.bfloat16)
        room, out = between(torch.full((R, N), 3e38, dtype=FP32, device=DEV), -3e38)
        moe.moe_linear_mx4(x, wq, ws, o, out=out)
        assert (room[:GUARD] == -3e38).all() and (room[-GUARD:] == -3e38).all() and torch.isfinite(out).all()
    assert all(torch.equal(h[0], b) for h, b in zip(held, before))


@pytest.mark.parametrize("R,N,K", [(1, 264, 1344), (5, 264, 1344), (300, 520, 1056), (4099, 4096, 1056)])
def test_dense_between_others(R, N, K):
    import bit_grouped_gemm_amd as moe
    print("test_dense_between_others", R, N, K, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(R)
    codes = lambda *s: torch.randint(0, 256, s, device=DEV, generator=g, dtype=torch.uint8)
    ones = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=DEV)
    xq, xs, wq, ws = (between(t, v)[1] for t, v in ((codes(R, K // 2), 0x77), (ones(R, K // 32), 255), (codes(N, K // 2), 0x77),
                                                   (ones(N, K // 32), 255)))
    room, out = between(torch.zeros(R, N, dtype=FP32, device=DEV), 9.0)
    moe.moe_mm_mx4(xq, xs, wq, ws, out=out)
    assert (room[:GUARD] == 9).all() and (room[-GUARD:] == 9).all()
    assert torch.equal(out, moe.moe_mm_mx4(*(t.clone() for t in (xq, xs, wq, ws)), out_dtype=FP32)) and torch.isfinite(out).all()
    x = between(torch.randn(R, K, device=DEV, generator=g).to(torch.bfloat16), float("nan"))[1]
    room, out = between(torch.zeros(R, N, dtype=FP32, device=DEV), 9.0)
    moe.moe_linear_mx4(x, wq, ws, out=out)
    assert (room[:GUARD] == 9).all() and (room[-GUARD:] == 9).all() and torch.isfinite(out).all()
