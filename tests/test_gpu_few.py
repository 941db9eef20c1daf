"""The few-token layer on 16-bit row-major weights against a plain 64-bit form
(needs an MI355X).

Tolerances.  The gate and up sums of H products, exact each, are off by at most
(H + 8) 2^-23 of the sum of their magnitudes; h = silu(g) u takes |u| 1.1 of the
gate's error, |silu(g)| of the up sum's and 8 roundings of its own, and is kept to
2^-17 of itself (bf16) or 2^-21 and 2^-24 (fp16).  The second sum carries that on with |W2| and
adds (I + 8) 2^-23 of its magnitudes, the weighted sum over slots 48 roundings,
the output type eps / 2 of the value.
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


def reference(x, ids, tw, w1, w2):
    """out and its error's bound, in 64 bits."""
    (T, H), (E, two, _), dt = x.shape, w1.shape, x.dtype
    I = two // 2
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    err, mag = torch.zeros_like(out), torch.zeros_like(out)
    keep, least = (2.0 ** -17, 0.0) if dt == BF16 else (2.0 ** -21, 2.0 ** -24)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        v, a, b = x[t].double(), w1[e].double(), w2[e].double()
        s, m = v @ a.t(), v.abs() @ a.abs().t() * (H + 8) * 2.0 ** -23
        gate, up = s[:, :I], s[:, I:]
        silu = gate * torch.sigmoid(gate)
        h = silu * up
        dh = 1.1 * up.abs() * m[:, :I] + silu.abs() * m[:, I:] + 1.1 * m[:, :I] * m[:, I:] + (8 * 2.0 ** -24 + keep) * h.abs() + least
        w = tw[t, j].double()[:, None]
        out.index_add_(0, t, w * (h @ b.t()))
        ym = h.abs() @ b.abs().t()
        err.index_add_(0, t, w.abs() * (dh @ b.abs().t() + (I + 8) * 2.0 ** -23 * ym))
        mag.index_add_(0, t, w.abs() * ym)
    return out, err + 48 * 2.0 ** -24 * mag


def check(got, ref, what):
    out, err = ref
    dt = got.dtype
    tol = err * 1.01 + torch.finfo(dt).eps / 2 * 1.01 * out.abs() + (2.0 ** -25 if dt == FP16 else 1e-38)
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - out).abs() / tol).max().item() if got.numel() else 0.0
    assert worst <= 1.0, (what, worst)


def route(g, T, E, k):
    score = torch.rand(T, E, device=DEV, generator=g)
    top = score.topk(k, 1)
    return top.indices.to(torch.int32), torch.softmax(top.values * 4, 1)


# (T, topk, E, H, I): one token; rows that fill no fragment, one, two, four; odd sizes; K shorter than a step and than a wave's share
SHAPES = [(1, 1, 1, 8, 8), (1, 8, 64, 512, 264), (1, 2, 8, 4096, 1408), (3, 2, 5, 72, 40), (7, 2, 8, 256, 128),
          (16, 1, 1, 264, 136), (17, 2, 3, 520, 72), (33, 2, 2, 328, 200), (64, 1, 1, 1032, 72), (64, 8, 64, 256, 512),
          (61, 8, 16, 1000, 328), (19, 6, 40, 2048, 1032), (5, 32, 33, 136, 64), (64, 32, 128, 64, 24), (2, 4, 1024, 64, 16),
          (9, 3, 6, 40, 2056), (64, 2, 2, 4096, 104)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,H,I", SHAPES)
def test_layer(T, k, E, H, I, dtype):
    moe = M()
    note("test_layer", T, k, E, H, I, dtype)
    g = gen(T * 7 + H + I)
    x = rand(g, T, H, dtype=dtype)
    w1, w2 = rand(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5), rand(g, E, H, I, dtype=dtype, scale=I ** -0.5)
    ids, tw = route(g, T, E, k)
    got = moe.moe_layer_mm(x, ids, tw, w1, w2)
    assert got.dtype == dtype and got.shape == (T, H)
    check(got, reference(x, ids, tw, w1, w2), "routed")
    # a second call on the same workspace, filled with anything, gives the same bits
    ws = torch.full((moe.moe_layer_mm_workspace_size(T, H, I, E, k),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws), got)
    assert torch.equal(moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws), got)
    # masked slots, everything on one expert, every token the same experts
    masked = torch.where(torch.rand(T, k, device=DEV, generator=g) < 0.5, torch.randint(0, 2, (T, k), device=DEV, generator=g, dtype=torch.int32) * (E + 1) - 1, ids)
    check(moe.moe_layer_mm(x, masked, tw, w1, w2, ws=ws), reference(x, masked, tw, w1, w2), "masked")
    same = ids[:1].expand(T, k).contiguous()
    check(moe.moe_layer_mm(x, same, tw, w1, w2, ws=ws), reference(x, same, tw, w1, w2), "same")


def test_no_slot_at_all():
    moe = M()
    g = gen(1)
    x, w1, w2 = rand(g, 9, 64), rand(g, 4, 32, 64), rand(g, 4, 64, 16)
    ids, tw = torch.full((9, 2), -1, dtype=torch.int32, device=DEV), torch.ones(9, 2, device=DEV)
    assert not moe.moe_layer_mm(x, ids, tw, w1, w2).any()
    ids[4, 1] = 3
    got = moe.moe_layer_mm(x, ids, tw, w1, w2)
    assert got[4].any() and not got[:4].any() and not got[5:].any()
    ids[:] = torch.tensor([-(1 << 31), (1 << 31) - 1], dtype=torch.int32)
    assert not moe.moe_layer_mm(x, ids, tw, w1, w2).any()
    assert moe.moe_layer_mm(x[:0], ids[:0], tw[:0], w1, w2).shape == (0, 64)


@pytest.mark.parametrize("T,k", [(5, 4), (64, 4), (64, 32)])
def test_a_token_that_names_an_expert_twice(T, k):
    """All slots on two experts: several tiles of one expert, and a token's rows in one tile."""
    moe = M()
    g = gen(2)
    x, w1, w2 = rand(g, T, 136), rand(g, 3, 80, 136, scale=0.1), rand(g, 3, 136, 40, scale=0.2)
    ids = torch.randint(0, 2, (T, k), device=DEV, generator=g, dtype=torch.int32) * 2
    tw = torch.rand(T, k, device=DEV, generator=g)
    check(moe.moe_layer_mm(x, ids, tw, w1, w2), reference(x, ids, tw, w1, w2), "twice")


def test_not_finite_stays_in_its_token():
    moe = M()
    g = gen(3)
    x, w1, w2 = rand(g, 40, 264), rand(g, 8, 144, 264, scale=0.06), rand(g, 8, 264, 72, scale=0.1)
    ids, tw = route(g, 40, 8, 2)
    clean = moe.moe_layer_mm(x, ids, tw, w1, w2)
    x[3, 100], x[17, 0] = float("nan"), float("inf")
    got = moe.moe_layer_mm(x, ids, tw, w1, w2)
    keep = [t for t in range(40) if t not in (3, 17)]
    assert torch.equal(got[keep], clean[keep])
    assert got[3].isnan().all() and not torch.isfinite(got[17]).any()
    # an expert that nobody names is not read into anything
    x[3, 100], x[17, 0] = 0, 0
    ids = torch.where(ids == 5, 4, ids)
    clean = moe.moe_layer_mm(x, ids, tw, w1, w2)
    w1[5], w2[5] = float("nan"), float("nan")
    assert torch.equal(moe.moe_layer_mm(x, ids, tw, w1, w2), clean)


def test_values_past_fp16():
    """h past fp16's range is infinite, in its token alone; just below it is exact."""
    moe = M()
    g = gen(4)
    x = torch.zeros(2, 64, dtype=FP16, device=DEV)
    x[0, 0], x[1, 0] = 240, 300
    w1 = torch.zeros(1, 16, 64, dtype=FP16, device=DEV)
    w1[0, 0, 0] = w1[0, 8, 0] = 1  # gate 0 and up 0: h = 240^2 = 57600, 300^2 = 90000
    w2 = torch.zeros(1, 64, 8, dtype=FP16, device=DEV)
    w2[0, 0, 0] = 2.0 ** -6
    got = moe.moe_layer_mm(x, torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, 1, device=DEV), w1, w2)
    assert got[0, 0] == 900 and not got[0, 1:].any()
    assert not torch.isfinite(got[1, 0])


def test_matrices_past_32_bits():
    """Weights of more than 2^32 bytes: the last experts'."""
    moe = M()
    g = gen(5)
    E, H, I = 40, 4096, 8200
    w1 = torch.zeros(E, 2 * I, H, dtype=BF16, device=DEV)
    w2 = torch.zeros(E, H, I, dtype=BF16, device=DEV)
    for e in (0, E - 1):
        w1[e] = rand(g, 2 * I, H, scale=0.015)
        w2[e] = rand(g, H, I, scale=0.01)
    assert w1.numel() * 2 > 1 << 32
    x = rand(g, 3, H)
    ids = torch.tensor([[E - 1, 0], [0, -1], [E - 1, 1]], dtype=torch.int32, device=DEV)
    tw = torch.rand(3, 2, device=DEV, generator=g)
    check(moe.moe_layer_mm(x, ids, tw, w1, w2), reference(x, ids, tw, w1, w2), "large")


def test_into_the_callers_tensor():
    moe = M()
    g = gen(6)
    x, w1, w2 = rand(g, 6, 72), rand(g, 4, 80, 72, scale=0.1), rand(g, 4, 72, 40, scale=0.1)
    ids, tw = route(g, 6, 4, 2)
    want = moe.moe_layer_mm(x, ids, tw, w1, w2)
    room = torch.full((8, 72), 5.0, dtype=BF16, device=DEV)
    got = moe.moe_layer_mm(x, ids, tw, w1, w2, out=room[1:7])
    assert torch.equal(room[1:7], want) and (room[::7] == 5).all() and got.data_ptr() == room[1:].data_ptr()
    long_ids, long_tw = torch.zeros(13, dtype=torch.int32, device=DEV), torch.zeros(13, device=DEV)
    long_ids[1:] = ids.reshape(-1)
    long_tw[1:] = tw.reshape(-1)
    assert torch.equal(moe.moe_layer_mm(x, long_ids[1:].view(6, 2), long_tw[1:].view(6, 2), w1, w2), want)  # 4-byte aligned
    with pytest.raises(moe.MoeError, match="65|unsupported|combination"):
        moe.moe_layer_mm(rand(g, 65, 72), *route(g, 65, 4, 2), w1, w2)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_mm(x, ids, tw, w1, w2, ws=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_streams_and_graph():
    moe = M()
    g = gen(7)
    w1, w2 = rand(g, 16, 528, 520, scale=0.04), rand(g, 16, 520, 264, scale=0.06)
    x = rand(g, 20, 520)
    ids, tw = route(g, 20, 16, 4)
    want = moe.moe_layer_mm(x, ids, tw, w1, w2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for k in range(6):  # two calls at once, each with scratch of its own
        with torch.cuda.stream(streams[k % 2]):
            outs.append(moe.moe_layer_mm(x, ids, tw, w1, w2))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = moe.moe_layer_mm(x, ids, tw, w1, w2)
    for k in range(4):
        x.copy_(rand(g, 20, 520))
        i2, t2 = route(g, 20, 16, 4)
        ids.copy_(i2)
        tw.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, moe.moe_layer_mm(x, ids, tw, w1, w2)), k


# widths whose columns leave CUs idle, with work enough that workgroups share them; k slots, eight waves and the
# workgroups of a column (8 at most here) are within the 48 roundings of `reference`
SHARED = [(1, 8, 8, 1024, 4096), (8, 8, 32, 2048, 512), (8, 3, 9, 520, 4000), (9, 8, 16, 2056, 520), (40, 8, 16, 2048, 512),
          (64, 4, 64, 1000, 328), (64, 32, 40, 1024, 264), (19, 8, 8, 12296, 264)]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,H,I", SHARED)
def test_shared_columns(T, k, E, H, I, dtype):
    moe = M()
    note("test_shared_columns", T, k, E, H, I, dtype)
    g = gen(T * 31 + k * 7 + E + H + I)
    x = rand(g, T, H, dtype=dtype)
    w1, w2 = rand(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5), rand(g, E, H, I, dtype=dtype, scale=I ** -0.5)
    ids, tw = route(g, T, E, k)
    got = moe.moe_layer_mm(x, ids, tw, w1, w2)
    check(got, reference(x, ids, tw, w1, w2), "routed")
    ws = torch.full((moe.moe_layer_mm_workspace_size(T, H, I, E, k),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws), got)
    same = ids[:1].expand(T, k).contiguous()
    check(moe.moe_layer_mm(x, same, tw, w1, w2, ws=ws), reference(x, same, tw, w1, w2), "same")
    # one slot only, then none: most workgroups have few steps, or none
    ids = torch.full_like(ids, -1)
    ids[T // 2, k // 2] = E - 1
    one = moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws)
    check(one, reference(x, ids, tw, w1, w2), "one slot")
    assert one[T // 2].any() and not one[:T // 2].any() and not one[T // 2 + 1:].any()
    ids[T // 2, k // 2] = E
    assert not moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws).any()


def test_shared_columns_in_a_graph():
    moe = M()
    g = gen(77)
    T, k, E, H, I = 40, 8, 16, 2048, 512
    x, w1, w2 = rand(g, T, H), rand(g, E, 2 * I, H, scale=H ** -0.5), rand(g, E, H, I, scale=I ** -0.5)
    ids, tw = route(g, T, E, k)
    out = torch.empty_like(x)
    ws = torch.empty(moe.moe_layer_mm_workspace_size(T, H, I, E, k), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_layer_mm(x, ids, tw, w1, w2, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_layer_mm(x, ids, tw, w1, w2, out=out, ws=ws)
    for i in range(4):
        x.copy_(rand(g, T, H))
        new_ids, new_tw = route(g, T, E, k)
        ids.copy_(new_ids)
        tw.copy_(new_tw)
        want = moe.moe_layer_mm(x, ids, tw, w1, w2)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
