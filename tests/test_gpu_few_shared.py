"""The few-token layer where workgroups share the columns of the second product and
have more than one column each: the end of one, whole ones, the beginning of
another (needs an MI355X; that each case is one, is checked in
test_few_shared_cpu.py).

Tolerances as in the other tests of the layer: a column's sums come from k slots,
eight waves and at most three workgroups here, within the 48 roundings that they
leave for that.
"""
import pytest
import torch

from test_gpu_few import BF16, FP16, DEV, check, gen, rand, reference, route

pytestmark = pytest.mark.gpu

# (T, topk, E, H, I, columns of a workgroup, rounded down): 16 columns of out at a time up to 8 tokens, 32 from there on
CASES = [(19, 8, 8, 12296, 2048, 1), (5, 8, 8, 4104, 2056, 1), (17, 8, 8, 8200, 1032, 1), (1, 8, 64, 5120, 1536, 1),
         (61, 8, 64, 12288, 1024, 1), (33, 2, 9, 8232, 776, 1), (64, 8, 16, 9000, 520, 1), (17, 8, 8, 16424, 1032, 2),
         (20, 4, 8, 24600, 1032, 3), (12, 8, 8, 8456, 1032, 1)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,H,I,columns", CASES)
def test_several_columns_a_workgroup(T, k, E, H, I, columns, dtype):
    import bit_grouped_gemm_amd as moe
    print("test_several_columns_a_workgroup", T, k, E, H, I, dtype, flush=True)
    g = gen(T * 31 + k * 7 + E + H + I)
    x = rand(g, T, H, dtype=dtype)
    w1, w2 = rand(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5), rand(g, E, H, I, dtype=dtype, scale=I ** -0.5)
    ids, tw = route(g, T, E, k)
    room = torch.full((T + 2, H), 5.0, dtype=dtype, device=DEV)
    ws = torch.full((moe.moe_layer_mm_workspace_size(T, H, I, E, k),), 255, dtype=torch.uint8, device=DEV)
    got = moe.moe_layer_mm(x, ids, tw, w1, w2, out=room[1:-1], ws=ws).clone()
    assert (room[0] == 5).all() and (room[-1] == 5).all()
    check(got, reference(x, ids, tw, w1, w2), "routed")
    for _ in range(3):  # the same bits every time, on a workspace that holds the last call's sums
        assert torch.equal(moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws), got)
    # few experts, so that a column has fewer steps than there are waves and workgroups; then one slot, then none
    same = ids[:1].expand(T, k).contiguous()
    same[:, 1:] = -1
    check(moe.moe_layer_mm(x, same, tw, w1, w2, ws=ws), reference(x, same, tw, w1, w2), "one expert")
    ids = torch.full_like(ids, -1)
    ids[T // 2, k // 2] = E - 1
    one = moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws)
    check(one, reference(x, ids, tw, w1, w2), "one slot")
    assert one[T // 2].any() and not one[:T // 2].any() and not one[T // 2 + 1:].any()
    ids[T // 2, k // 2] = E
    assert not moe.moe_layer_mm(x, ids, tw, w1, w2, ws=ws).any()


def test_in_a_graph():
    import bit_grouped_gemm_amd as moe
    g = gen(78)
    T, k, E, H, I, _ = CASES[2]
    x, w1, w2 = rand(g, T, H), rand(g, E, 2 * I, H, scale=H ** -0.5), rand(g, E, H, I, scale=I ** -0.5)
    ids, tw = route(g, T, E, k)
    out = torch.empty_like(x)
    ws = torch.empty(moe.moe_layer_mm_workspace_size(T, H, I, E, k), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
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
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
