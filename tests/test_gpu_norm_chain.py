"""The norm, the router, the few-token layer and the quantised products together,
as a block of a model uses them (needs an MI355X).

Every stage is held to its own plain 64-bit form on what the stage before it
gave, with that stage's tolerance: 48 roundings for a norm; (K + 8) 2^-23 of the
magnitudes and the output's rounding for a product; half a step of the format for
a quantised value.
"""
import sys

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
kN = 48 * 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M().load()
    yield


def M():
    import bit_grouped_gemm_amd as moe
    return moe


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
    worst = ((got.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, (what, worst)


def norm_ref(s, w):
    v = s.double()
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * w.double()


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def mx4_values(codes, scales):
    level = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    return level[c] * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def test_decode_block_on_16_bit_experts():
    """norm(x + residual) -> router -> the layer -> the next norm, two blocks in a row: stage by
    stage, and the whole run captured and replayed."""
    moe = M()
    g = gen(1)
    T, H, I, E, k = 11, 512, 264, 16, 4
    cfg = moe.Cfg(T, H, 128, E, k, moe.WFMT_FP8_BLOCK, 128, 128)  # the router's T, H, E and topk
    gate = [rand(g, E, H, scale=0.05) for _ in range(2)]
    w1 = [rand(g, E, 2 * I, H, scale=H ** -0.5) for _ in range(2)]
    w2 = [rand(g, E, H, I, scale=I ** -0.5) for _ in range(2)]
    nw = [rand(g, H, dtype=FP32) for _ in range(3)]
    x, res = rand(g, T, H), rand(g, T, H)

    def run():
        stages, out, stream = [], x, res
        for b in range(2):
            y, stream = moe.moe_rms_norm(out, nw[b], stream, eps=EPS)
            ids, tw = moe.moe_route(cfg, y, gate[b])
            out = moe.moe_layer_mm(y, ids, tw, w1[b], w2[b])
            stages.append((y, stream, ids, tw, out))
        y, stream = moe.moe_rms_norm(out, nw[2], stream, eps=EPS)
        return stages, y, stream

    stages, y, stream = run()
    before, total = x, res
    for b, (n, s, ids, tw, out) in enumerate(stages):
        assert torch.equal(s, (before.float() + total.float()).to(BF16))
        ref = norm_ref(s, nw[b])
        within(n, ref, kN * ref.abs() + rounding(ref, BF16) * 1.001, "norm")
        logits = n.double() @ gate[b].double().t()
        best = logits.topk(k, 1)
        wide = (n.double().abs() @ gate[b].double().abs().t()) * (H + 8) * 2.0 ** -23
        assert (logits.gather(1, ids.long()) >= best.values - 2 * wide.amax(1, keepdim=True)).all()
        want = torch.softmax(logits.gather(1, ids.long()), 1)
        within(tw, want, 4 * wide.amax(1, keepdim=True) * want + 32 * 2.0 ** -24 * want, "router")
        ref, err = torch.zeros(T, H, dtype=torch.float64, device=DEV), torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in range(E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if len(t):
                v, a, c = n[t].double(), w1[b][e].double(), w2[b][e].double()
                p, m = v @ a.t(), v.abs() @ a.abs().t() * (H + 8) * 2.0 ** -23
                silu = p[:, :I] * torch.sigmoid(p[:, :I])
                h = silu * p[:, I:]
                dh = 1.1 * p[:, I:].abs() * m[:, :I] + (silu.abs() + 1.1 * m[:, :I]) * m[:, I:] + 2.0 ** -16 * h.abs()
                wt = tw[t, j].double()[:, None]
                ref.index_add_(0, t, wt * (h @ c.t()))
                err.index_add_(0, t, wt * (dh @ c.abs().t() + (I + 64) * 2.0 ** -23 * (h.abs() @ c.abs().t())))
        within(out, ref, err * 1.01 + rounding(ref, BF16), "layer")
        before, total = out, s
    ref = norm_ref(stream, nw[2])
    within(y, ref, kN * ref.abs() + rounding(ref, BF16) * 1.001, "last norm")

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        kept = run()
    for i in range(3):
        x.copy_(rand(g, T, H))
        res.copy_(rand(g, T, H))
        graph.replay()
        torch.cuda.synchronize()
        got = kept[1].clone(), kept[2].clone()
        eager = run()
        assert torch.equal(got[0], eager[1]) and torch.equal(got[1], eager[2]), i


@pytest.mark.parametrize("group", [32, 128])
def test_norm_codes_into_the_layers_first_product(group):
    """The norm's e4m3 codes and scales in the place of moe_permute's, on both of the layer's block sizes."""
    moe = M()
    g = gen(2)
    wl = synth.WORKLOADS["decode_fp8"].with_shape(H=512, I=256, E=8, topk=2, wblk=group, act_group=group)
    T = 21
    cfg = moe.Cfg.for_workload(wl, T)
    weights = synth.gen_weights(wl, seed=0, device=DEV)
    packed = moe.moe_prepack_weights(cfg, weights)
    x, res, nw = rand(g, T, wl.H), rand(g, T, wl.H), rand(g, wl.H, dtype=FP32)
    codes, scales, y, s = moe.moe_rms_norm_quant(x, nw, res, eps=EPS, fmt=moe.QFMT_E4M3, group=group, want_y=True)
    ids, tw = moe.moe_route(cfg, y, rand(g, wl.E, wl.H, scale=0.05))
    counts, offsets, eidx, rtok, xq, xs = moe.moe_permute(cfg, y, ids)
    # the same codes as the layer's own quantiser's, but where y's rounding to bf16 crosses a border
    assert codes.shape == xq.shape and scales.shape == xs.shape
    assert ((scales / xs - 1).abs() <= 2.0 ** -8).all() and (codes != xq).double().mean() < 0.1
    hq, hs = moe.moe_grouped_gemm1_swiglu(cfg, codes, scales, rtok, offsets, packed)
    v = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(group, 1)
    h = hq.view(torch.float8_e4m3fn).double() * hs.double().repeat_interleave(group, 1)
    o = offsets.tolist()
    for e in range(wl.E):
        if o[e] == o[e + 1]:
            continue
        w1 = weights.w1[e].view(torch.float8_e4m3fn).double()
        w1 = w1 * weights.w1s[e].double().repeat_interleave(group, 0).repeat_interleave(group, 1)
        rows = rtok[o[e]:o[e + 1]].long()
        p = v[rows] @ w1.t()
        m = (v[rows].abs() @ w1.abs().t()) * (wl.H + 8) * 2.0 ** -23
        gate, up = p[:, :wl.I], p[:, wl.I:]
        silu = gate * torch.sigmoid(gate)
        ref = silu * up
        off = 1.1 * up.abs() * m[:, :wl.I] + (silu.abs() + m[:, :wl.I]) * m[:, wl.I:] + 8 * 2.0 ** -24 * ref.abs()
        unit = hs[o[e]:o[e + 1]].double().repeat_interleave(group, 1)
        half = torch.maximum(2.0 ** -4 * ref.abs(), unit * 2.0 ** -10)
        within(h[o[e]:o[e + 1]], ref, half * 1.001 + off * 1.01, "h")


def test_norm_codes_into_the_int8_and_mxfp4_products():
    moe = M()
    g = gen(3)
    R, K, N = 70, 1056, 392
    x, res, nw = rand(g, R, K), rand(g, R, K), rand(g, K, dtype=FP32)
    w = rand(g, N, K, scale=0.05)
    codes, scales, _, s = moe.moe_rms_norm_quant(x, nw, res, eps=EPS, fmt=moe.QFMT_I8)
    wq, ws = moe.moe_quant_i8(w)
    got = moe.moe_mm_i8(codes, scales, wq, ws, out_dtype=FP32)
    ref = (codes.double() @ wq.double().t()) * scales.double()[:, None] * ws.double()
    within(got, ref, 4 * 2.0 ** -24 * ref.abs() + 1e-30, "int8")
    codes, scales, _, s2 = moe.moe_rms_norm_quant(x, nw, res, eps=EPS, fmt=moe.QFMT_MXFP4)
    assert torch.equal(s, s2)
    wq, ws = moe.moe_quant_mx4(w)
    got = moe.moe_mm_mx4(codes, scales, wq, ws)
    a, b = mx4_values(codes, scales), mx4_values(wq, ws)
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    within(got, ref, (K + 8) * 2.0 ** -23 * mag + rounding(ref, BF16), "mxfp4")


def test_quantiser_is_the_layers():
    """moe_quant_mx4 and the 4-bit layer's own activation quantiser: the same codes and scales."""
    moe = M()
    g = gen(4)
    for T, H in ((1, 256), (37, 512), (300, 4096)):
        cfg = moe.Cfg(T, H, 256, 8, 2, moe.WFMT_MXFP4, 32, 32, 0, 1)
        x = rand(g, T, H)
        x[0, :64] = 0
        ids = torch.zeros(T, 2, dtype=torch.int32, device=DEV)
        _, _, _, _, xq, xs = moe.moe_permute(cfg, x, ids)
        codes, scales = moe.moe_quant_mx4(x)
        assert torch.equal(xq, codes) and torch.equal(xs, scales)


def test_mxfp4_experts_without_prepacking():
    """Routing, the gate|up product, SwiGLU with the down product, the combine: MXFP4 experts that
    moe_quant_mx4 made of 16-bit weights, on the layer's permute and combine."""
    moe = M()
    g = gen(5)
    T, H, I, E, k = 45, 512, 256, 8, 2
    cfg = moe.Cfg(T, H, I, E, k, moe.WFMT_FP8_BLOCK, 128, 128)
    x = rand(g, T, H)
    ids, tw = moe.moe_route(cfg, x, rand(g, E, H, scale=0.05))
    _, offsets, eidx, rtok, _, _ = moe.moe_permute(cfg, x, ids)
    q1, s1 = moe.moe_quant_mx4(rand(g, E * 2 * I, H, scale=0.05))
    q2, s2 = moe.moe_quant_mx4(rand(g, E * H, I, scale=0.05))
    q1, s1, q2, s2 = q1.view(E, 2 * I, -1), s1.view(E, 2 * I, -1), q2.view(E, H, -1), s2.view(E, H, -1)
    gu = moe.moe_linear_mx4(x, q1, s1, offsets, row_token=rtok)
    y = moe.moe_linear_mx4(gu, q2, s2, offsets, swiglu=True, out_dtype=FP32)
    out = moe.moe_combine(cfg, y, eidx, offsets, tw)
    a = mx4_values(*moe.moe_quant_mx4(x))
    hq = mx4_values(*moe.moe_quant_mx4(gu, swiglu=True))
    o = offsets.tolist()
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        v, w1, w2 = a[rtok[lo:hi].long()], mx4_values(q1[e], s1[e]), mx4_values(q2[e], s2[e])
        ref = v @ w1.t()
        if hi > lo:
            within(gu[lo:hi], ref, (H + 8) * 2.0 ** -23 * (v.abs() @ w1.abs().t()) + rounding(ref, BF16), "gate|up")
            ref = hq[lo:hi] @ w2.t()
            within(y[lo:hi], ref, (I + 8) * 2.0 ** -23 * (hq[lo:hi].abs() @ w2.abs().t()) + 1e-30, "down")
    ref = (y.double()[eidx.long().view(T, k)] * tw.double()[:, :, None]).sum(1)
    mag = (y.double().abs()[eidx.long().view(T, k)] * tw.double()[:, :, None]).sum(1)
    within(out, ref, 8 * 2.0 ** -24 * mag + rounding(ref, BF16), "combine")


def test_training_block():
    """norm -> grouped products of one expert layer, gradients through both norms' inputs and weights:
    the chain's gradients against those that autograd makes of the same steps in 64 bits."""
    moe = M()
    g = gen(6)
    R, K, N, E = 130, 264, 136, 3
    x, res = rand(g, R, K).requires_grad_(), rand(g, R, K).requires_grad_()
    nw = (1 + 0.1 * torch.randn(K, device=DEV, generator=g)).requires_grad_()
    w = rand(g, E, N, K, scale=0.05).requires_grad_()
    o = torch.tensor([0, 50, 50, R], dtype=torch.int32, device=DEV)
    y, s = moe.moe_rms_norm(x, nw, res, eps=EPS)
    z = moe.moe_grouped_mm(y, w, o)
    dz, ds = rand(g, R, N), rand(g, R, K)
    got = torch.autograd.grad((z, s), (x, res, nw, w), (dz, ds))
    # the same steps with the values that the chain rounded: y's gradient is rounded to bf16 between
    dy = moe.moe_grouped_mm_dgrad(dz, w.detach(), o)
    v = s.detach().double()
    rstd = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
    n, gr = v * rstd, dy.double() * nw.detach().double()
    ref = rstd * (gr - n * (gr * n).mean(1, keepdim=True)) + ds.double()
    mag = rstd * (gr.abs() + n.abs() * (gr * n).abs().mean(1, keepdim=True)) + ds.double().abs()
    within(got[0], ref, 128 * 2.0 ** -24 * mag + rounding(ref, BF16), "dx")
    assert torch.equal(got[0], got[1])
    within(got[2], (dy.double() * n).sum(0), 200 * 2.0 ** -24 * (dy.double() * n).abs().sum(0) + 1e-30, "dweight")
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
    mg = torch.zeros_like(dw)
    for e, (a, b) in enumerate(((0, 50), (50, 50), (50, R))):
        dw[e] = dz[a:b].double().t() @ y[a:b].detach().double()
        mg[e] = dz[a:b].double().abs().t() @ y[a:b].detach().double().abs()
    within(got[3], dw, (R + 8) * 2.0 ** -23 * mg + rounding(dw, BF16), "dw")
