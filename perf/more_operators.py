"""Cases of the operators around the expert products: the root-mean-square norm
with the residual's addition, its quantised form and its gradients; the MXFP4
product on row-major weights; the whole expert layer for a few tokens on 16-bit
row-major weights.

Shapes are those of the MoE layers of this repository (H=4096, E=64, top-8,
I=1536; H=7168, I=2048; the tiny H=256, E=8, I=128 layer) and generic ones
around them.  Rows come from a top-k routing of T tokens: expert popularity
falls as rank^-skew (0 is uniform), so groups are ragged and some stay empty.

Kinds of cases
  norm    s = x + residual, y = s / rms(s) * weight, in 16 bits
  norm_q  the same with y's e4m3 codes and one scale per `group` channels
  step    norm and its backward pass: y, s, dx (the residual's gradient too) and dweight
  linear  16-bit activations (through SwiGLU where `swiglu`) quantised to MXFP4,
          times MXFP4 weights: dense (E = 0) or grouped by expert
  mm      the MXFP4 product with the codes in hand, rows gathered from tokens
  layer   out[t] = sum_j weight[t][j] * W2_e (silu(G) * U), (G, U) = W1_e x[t], e = id[t][j];
          `elsewhere`: the share of experts that another GPU holds (their slots are masked)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the norm in front of a decoded token's router: one row, bound by latency
        dict(name="norm_one_token_bf16", kind="norm", R=1, K=4096, dtype="bf16", residual=True),
        # a decode batch of 61 sequences on its way into the fp8 layer, the router's rows beside the codes
        dict(name="norm_q_decode_bf16", kind="norm_q", R=61, K=7168, dtype="bf16", residual=True, group=128),
        # a prompt of 4099 tokens, scales per 32 channels
        dict(name="norm_q_prefill_fp16", kind="norm_q", R=4099, K=4096, dtype="fp16", residual=True, group=32),
        # a training step's norm, forward and backward, in a residual stream
        dict(name="step_bf16", kind="step", R=16384, K=4096, dtype="bf16", residual=True),
        # one token through a dense MXFP4 projection (a shared expert's): bound by the weights' bytes
        dict(name="linear_one_token_bf16", kind="linear", T=1, topk=1, E=0, K=7168, N=4096, dtype="bf16",
             swiglu=False, skew=0.0),
        # the down projection of a decode batch: SwiGLU, quantisation and the grouped product
        dict(name="linear_decode_swiglu_bf16", kind="linear", T=61, topk=8, E=64, K=2048, N=7168, dtype="bf16",
             swiglu=True, skew=0.5),
        # a prompt through a dense projection
        dict(name="linear_prefill_fp16", kind="linear", T=4099, topk=1, E=0, K=7168, N=4096, dtype="fp16",
             swiglu=False, skew=0.0),
        # a prompt of 4096 tokens, gathered to the experts' rows, to fp32
        dict(name="mm_prefill_fp32", kind="mm", T=4096, topk=8, E=64, K=4096, N=1536, dtype="fp32", skew=0.3),
        # the tiny layer, seven tokens: bound by latency
        dict(name="layer_tiny_fp16", kind="layer", T=7, topk=2, E=8, H=256, I=128, dtype="fp16", skew=0.0,
             elsewhere=0.0),
        # decoding one token through 8 of 64 experts: bound by the weights' bytes
        dict(name="layer_one_token_bf16", kind="layer", T=1, topk=8, E=64, H=4096, I=1408, dtype="bf16", skew=0.0,
             elsewhere=0.0),
        # a decode batch on one of two GPUs that share the experts, popular ones hit more often
        dict(name="layer_decode_fp16", kind="layer", T=19, topk=8, E=32, H=7168, I=2048, dtype="fp16", skew=0.5,
             elsewhere=0.5),
        # a larger decode batch: every expert has rows
        dict(name="layer_batch_bf16", kind="layer", T=61, topk=8, E=64, H=4096, I=1408, dtype="bf16", skew=0.3,
             elsewhere=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["norm", "norm_q", "step", "linear", "mm", "layer"])
    if kind in ("norm", "norm_q", "step"):
        group = rng.choice([32, 128])
        K = _log_int(rng, 128, 8192, group if kind == "norm_q" else 8)
        R = _log_int(rng, 1, min(16384, (1 << 26) // K))
        c = dict(kind=kind, R=R, K=K, dtype=rng.choice(["bf16", "fp16"]), residual=rng.random() < 0.7)
        if kind == "norm_q":
            c["group"] = group
        return c
    if kind == "layer":
        H, I = _log_int(rng, 128, 7168, 8), _log_int(rng, 64, 2048, 8)
        E = rng.randint(1, max(1, min(64, (1 << 30) // (2 * H * I))))
        return dict(kind=kind, T=_log_int(rng, 1, 64), topk=rng.randint(1, min(8, E)), E=E, H=H, I=I,
                    dtype=rng.choice(["bf16", "fp16"]), skew=rng.choice([0.0, 0.5, 1.2]),
                    elsewhere=rng.choice([0.0, 0.0, 0.5]))
    K, N = _log_int(rng, 128, 7168, 32), _log_int(rng, 128, 4096, 8)
    E = rng.choice([0, rng.randint(2, 64)])
    topk = rng.randint(1, min(8, max(1, E)))
    rows = _log_int(rng, 1, int(max(1, min(32768, 2e11 / (K * N)))))
    c = dict(kind=kind, T=max(1, rows // topk), topk=topk, E=E, K=K, N=N, skew=rng.choice([0.0, 0.5, 1.2]))
    c["dtype"] = rng.choice(["bf16", "fp16", "fp32"]) if kind == "mm" else rng.choice(["bf16", "fp16"])
    if kind == "linear":
        c["swiglu"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _popularity(case, E):
    p = [(e + 1) ** -case["skew"] for e in range(E)]
    s = sum(p)
    return [v / s for v in p]


def _choose(case, E, g):
    """The scores and numbers of the topk of E experts that each token takes."""
    p = torch.tensor(_popularity(case, E), device="cuda")
    noise = -torch.rand(case["T"], E, device="cuda", generator=g).clamp_min(1e-20).log()
    top = (p.log() - noise.log()).topk(case["topk"], dim=1)
    return top.values, top.indices


def _groups(ids, E):
    """offsets int32 [E + 1], the slots in the order of their experts, and the largest group."""
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offsets, order, int(counts.max())


def _randn(shape, scale, dtype, g):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.reshape(-1).split(1 << 26):
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) * scale)
    return out


def _pack(v, exponent):
    """Two e2m1 codes per byte (even column in the low half) and the e8m0 bytes of quantised values."""
    mag = (v.abs() * 2).to(torch.int64)  # 0 1 2 3 4 6 8 12: the codes' magnitudes, doubled
    code = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], device=v.device)[mag] + 8 * (v < 0)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), (exponent + 127).to(torch.uint8)


def _weights_mx4(E, N, K, g):
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _pack(*_plain_quant(torch.randn(N, K, device="cuda", generator=g) * 0.02))
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    s, kind, dt = dict(case), case["kind"], DTYPES[case["dtype"]]
    if kind in ("norm", "norm_q", "step"):
        R, K = case["R"], case["K"]
        # tokens differ in size, as rows of a residual stream do, and a few channels stand out
        size = torch.exp(torch.randn(R, 1, device="cuda", generator=g) * 0.5)
        channel = torch.exp(torch.randn(K, device="cuda", generator=g) * 0.7)
        s["x"] = (torch.randn(R, K, device="cuda", generator=g) * size * 0.5).to(dt)
        s["res"] = (torch.randn(R, K, device="cuda", generator=g) * size * channel).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(dt)
        if kind == "step":
            s["dy"] = _randn((R, K), 0.05, dt, g)
            s["ds"] = _randn((R, K), 0.05, dt, g) if case["residual"] else None
            for n in ("x", "res", "weight"):
                if s[n] is not None:
                    s[n].requires_grad_()
        return s
    T, k, E = case["T"], case["topk"], case["E"]
    if kind == "layer":
        H, I = case["H"], case["I"]
        # E experts are here, as many more as `elsewhere` says on other GPUs
        total = round(E / (1 - case["elsewhere"]))
        score, ids = _choose(case, total, g)
        here = torch.randperm(total, device="cuda", generator=g)  # the experts' places
        ids = here[ids]
        s["topk_ids"] = torch.where(ids < E, ids, -1).to(torch.int32)
        s["topk_weights"] = torch.softmax(score, dim=1)
        s["x"] = _randn((T, H), 1.0, dt, g)
        s["w1"] = _randn((E, 2 * I, H), 0.02, dt, g)
        s["w2"] = _randn((E, H, I), 0.02, dt, g)
        s["most"] = _groups(ids.reshape(-1).clamp_max(E), E + 1)[2]
        return s
    K, N = case["K"], case["N"]
    if E:
        s["offsets"], order, s["most"] = _groups(_choose(case, E, g)[1].reshape(-1), E)
        s["row_token"] = (order // k).to(torch.int32)
    s["wq"], s["ws"] = _weights_mx4(max(1, E), N, K, g)
    if not E:
        s["wq"], s["ws"] = s["wq"][0], s["ws"][0]
    if kind == "linear":
        size = torch.exp(torch.randn(T * k, 1, device="cuda", generator=g) * 0.5)
        s["x"] = (torch.randn(T * k, 2 * K if case["swiglu"] else K, device="cuda", generator=g) * size).to(dt)
    else:
        s["xq"], s["xs"] = _pack(*_plain_quant(torch.randn(T, K, device="cuda", generator=g)))
    return s


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    x = s["x"].detach()
    total = x if s["res"] is None else (x.float() + s["res"].detach().float()).to(x.dtype)
    v = total.float()
    rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    return total, v * rstd, rstd


def _plain_step(s):
    total, n, rstd = _plain_norm(s)
    dt, w, dy = total.dtype, s["weight"].detach().float(), s["dy"].float()
    g = dy * w
    dx = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    dw = (dy * n).sum(dim=0)
    y = (n * w).to(dt)
    if s["res"] is None:
        return y, dx.to(dt), dw.to(dt)
    dx = (dx + s["ds"].float()).to(dt)
    return y, total, dx, dx, dw.to(dt)


def _plain_norm_q(s):
    total, n, _ = _plain_norm(s)
    y, group = n * s["weight"].float(), s["group"]
    blocks = y.view(y.shape[0], -1, group)
    top = blocks.abs().amax(dim=2, keepdim=True).clamp_min(2.0 ** -64)
    mult = top.new_full((), 448.0) / top
    codes = (blocks * mult).clamp(-448, 448).to(torch.float8_e4m3fn).view(y.shape)
    return codes, mult.reciprocal()[:, :, 0], y.to(total.dtype), total


def _plain_quant(v):
    """Values on the e2m1 grid [R, K] and the exponents of their blocks' scales [R, K / 32], fp32."""
    blocks = v.view(v.shape[0], -1, 32)
    top = blocks.abs().amax(dim=2)
    exponent = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    exponent = torch.where(top == 0, -127, exponent)
    u = blocks * torch.exp2(-exponent.float())[:, :, None]  # (ldexp's powers are not exact on a GPU)
    a = u.abs()
    # steps of 1/2 below 2, of 1 below 4, of 2 above; ties to even
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(u / step) * step).clamp(-6, 6).view(v.shape), exponent


def _plain_values(codes, scales):
    """The fp32 values that packed codes [..., K / 2] and e8m0 bytes [..., K / 32] stand for."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    pairs = torch.arange(256, device=codes.device)
    both = torch.stack([table[pairs % 16], table[pairs // 16]], dim=1)  # byte -> its two values
    v = both[codes.int()].reshape(*scales.shape, 32)
    return (v * torch.exp2(scales.float() - 127)[..., None]).reshape(*codes.shape[:-1], -1)


def _slots(offsets, most, rows):
    """Place of each row in a [E, most] grid of rows: the groups padded to the largest one."""
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].contiguous(), r.to(offsets.dtype), right=True)
    return e * most + (r - offsets[e])


def _grouped(x, w, slots, most):
    """fp32 x[r] @ w[e]^T for the rows r of each group e."""
    E, N, K = w.shape
    xp = torch.zeros(E * most, K, dtype=torch.float32, device=x.device)
    xp[slots] = x.float()
    xt = xp.view(E, most, K).transpose(1, 2).contiguous()
    return torch.bmm(w.float(), xt).transpose(1, 2).reshape(E * most, N)[slots]


def _plain_product(s, x, dtype):
    w = _plain_values(s["wq"], s["ws"])
    if s["E"]:
        return _grouped(x, w, _slots(s["offsets"], s["most"], x.shape[0]), s["most"]).to(dtype)
    return (x @ w.t()).to(dtype)


def _plain_linear(s):
    v = s["x"].float()
    if s["swiglu"]:
        gate, up = v.chunk(2, dim=1)
        v = gate / (1 + torch.exp(-gate)) * up
    u, exponent = _plain_quant(v)
    x = u.view(*exponent.shape, 32) * torch.exp2(exponent.float())[:, :, None]
    return _plain_product(s, x.view(u.shape), s["x"].dtype)


def _plain_mm(s):
    x = _plain_values(s["xq"], s["xs"])
    return _plain_product(s, x[s["row_token"].long()] if s["E"] else x, DTYPES[s["dtype"]])


def _plain_layer(s):
    x, E, I, T, k = s["x"], s["E"], s["I"], s["T"], s["topk"]
    ids = s["topk_ids"].reshape(-1).long()
    mine = ids >= 0
    ids = torch.where(mine, ids, E)  # a group of its own behind the experts
    order = torch.sort(ids, stable=True).indices
    offsets = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=E + 1).cumsum(0)])
    slots, most = _slots(offsets, s["most"], T * k), s["most"]
    here = slots.clamp_max(E * most - 1)  # (rows of that group share the last expert's rows, and count for nothing)
    here = torch.where(slots < E * most, here, E * most)
    xp = torch.zeros(E * most + 1, x.shape[1], dtype=torch.float32, device=x.device)
    xp[here] = x.float()[order // k]
    xt = xp[:-1].view(E, most, -1).transpose(1, 2).contiguous()
    both = torch.bmm(s["w1"].float(), xt)  # [E, 2 I, most]
    gate, up = both[:, :I], both[:, I:]
    h = gate / (1 + torch.exp(-gate)) * up
    rows = torch.bmm(s["w2"].float(), h.contiguous()).transpose(1, 2).reshape(E * most, -1)
    y = torch.zeros(T * k, rows.shape[1], dtype=torch.float32, device=x.device)
    y[order] = rows[here.clamp_max(E * most - 1)]
    weight = torch.where(mine, s["topk_weights"].reshape(-1), 0.0)
    return (y * weight[:, None]).view(T, k, -1).sum(dim=1).to(x.dtype)


def _plain(s):
    kind = s["kind"]
    if kind == "norm":
        total, n, _ = _plain_norm(s)
        y = (n * s["weight"].float()).to(total.dtype)
        return y if s["res"] is None else (y, total)
    return {"norm_q": _plain_norm_q, "step": _plain_step, "linear": _plain_linear, "mm": _plain_mm,
            "layer": _plain_layer}[kind](s)


def run(state):
    if not own:
        return _plain(state)
    import bit_grouped_gemm_amd as moe
    s, kind = state, state["kind"]
    if kind == "norm":
        return moe.moe_rms_norm(s["x"], s["weight"], s["res"], eps=EPS)
    if kind == "norm_q":
        codes, scales, y, total = moe.moe_rms_norm_quant(s["x"], s["weight"], s["res"], eps=EPS, fmt=moe.QFMT_E4M3,
                                                         group=s["group"], want_y=True)
        return codes.view(torch.float8_e4m3fn), scales, y, s["x"] if total is None else total
    if kind == "step":
        if s["res"] is None:
            y = moe.moe_rms_norm(s["x"], s["weight"], eps=EPS)
            return y, *torch.autograd.grad(y, (s["x"], s["weight"]), s["dy"])
        y, total = moe.moe_rms_norm(s["x"], s["weight"], s["res"], eps=EPS)
        return y, total, *torch.autograd.grad((y, total), (s["x"], s["res"], s["weight"]), (s["dy"], s["ds"]))
    if kind == "linear":
        return moe.moe_linear_mx4(s["x"], s["wq"], s["ws"], s.get("offsets"), swiglu=s["swiglu"])
    if kind == "mm":
        return moe.moe_mm_mx4(s["xq"], s["xs"], s["wq"], s["ws"], s.get("offsets"), row_token=s.get("row_token"),
                              out_dtype=DTYPES[s["dtype"]])
    return moe.moe_layer_mm(s["x"], s["topk_ids"], s["topk_weights"], s["w1"], s["w2"])


def work(case):
    kind = case["kind"]
    if kind in ("norm", "norm_q", "step"):
        n, res = float(case["R"] * case["K"]), case["residual"]
        b = 2 * n * (4 if res else 2) + 2.0 * case["K"]  # x and the residual in, y and their sum out
        if kind == "norm_q":
            b += n + 4 * n / case["group"]
        if kind == "step":  # dy (and the sum's gradient) and the sum in again, dx out
            b += 2 * n * (4 if res else 3) + 4.0 * case["K"]
        return {"bytes": b, "flops": (16 if kind == "step" else 6) * n}
    T, k, E = case["T"], case["topk"], case["E"]
    total = round(E / (1 - case.get("elsewhere", 0.0)))
    # experts that get a row, each slot taken as a draw from the popularity
    touched = sum(1 - (1 - min(1.0, k * p)) ** T for p in _popularity(case, total)) * E / total if E else 1
    rows = T * k * (E / total if E else 1)
    touched = min(touched, rows)
    if kind == "layer":
        H, I = case["H"], case["I"]
        return {"bytes": 2.0 * (2 * T * H + touched * 3 * H * I) + 8.0 * T * k, "flops": 6.0 * rows * H * I}
    K, N = case["K"], case["N"]
    weights = touched * N * (K / 2 + K / 32)
    if kind == "linear":
        return {"bytes": 2.0 * rows * ((2 if case["swiglu"] else 1) * K + N) + weights, "flops": 2.0 * rows * K * N}
    out = 4.0 if case["dtype"] == "fp32" else 2.0
    return {"bytes": (T if E else rows) * (K / 2 + K / 32) + out * rows * N + weights, "flops": 2.0 * rows * K * N}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(case, s):
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    x, w = s["x"].detach().double(), s["weight"].detach().double()
    K = x.shape[1]
    total = x
    if s["res"] is not None:
        total = (x + s["res"].detach().double()).to(dt).double()
    r = torch.sqrt(total.square().sum(1) / K + EPS)
    y = torch.einsum("rk,r,k->rk", total, 1 / r, w)
    if kind == "norm":
        return y if s["res"] is None else (y, total)
    if kind == "norm_q":
        G = case["group"]
        scale = y.reshape(-1, G).abs().amax(1).clamp_min(2.0 ** -64) / 448
        q = (y.reshape(-1, G) / scale[:, None]).reshape(y.shape)
        # e4m3: three bits behind the first one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        codes = (torch.round(q / step) * step).clamp(-448, 448)
        return codes, scale.view(x.shape[0], -1), y, total
    # dL/ds_j = w_j dy_j / r - s_j (sum_i w_i dy_i s_i) / (K r^3)
    dy = s["dy"].double()
    inner = ((dy * w) * total).sum(1)
    dx = dy * w / r[:, None] - total * (inner / (K * r ** 3))[:, None]
    dw = ((dy * total) / r[:, None]).sum(0)
    if s["res"] is None:
        return y, dx, dw
    dx = dx + s["ds"].double()
    return y, total, dx, dx, dw


def _exact_e2m1(a):
    """The nearest of the e2m1 magnitudes, at a tie the one with the even code."""
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=a.device)
    middle = (level[1:] + level[:-1]) / 2
    below, above = torch.bucketize(a, middle), torch.bucketize(a, middle, right=True)
    return level[torch.where(below % 2 == 0, below, above)]


def _exact_quant(v):
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    power = torch.floor(torch.log2(top.clamp_min(2.0 ** -200))).clamp(-125, 129) - 2
    scale = torch.exp2(power)
    return (torch.sign(b) * _exact_e2m1(b.abs() / scale) * scale).reshape(v.shape)


def _exact_unpack(codes, scales):
    low, high = (codes & 15).long(), (codes >> 4).long()
    code = torch.stack([low, high], dim=-1).flatten(-2)
    mantissa, ex = (code & 1).double(), (code >> 1) & 3
    v = torch.where(ex == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2(ex.double() - 1))
    v = torch.where(code >= 8, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    kind, E = case["kind"], case["E"] if "E" in case else 0
    if kind in ("norm", "norm_q", "step"):
        return _exact_norm(case, s)
    if kind == "layer":
        I = case["I"]
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for e in range(E):
            t, j = torch.nonzero(s["topk_ids"] == e, as_tuple=True)
            if len(t) == 0:
                continue
            both = s["x"][t].double() @ s["w1"][e].double().t()
            h = both[:, :I] * torch.sigmoid(both[:, :I]) * both[:, I:]
            y = h @ s["w2"][e].double().t()
            out.index_add_(0, t, y * s["topk_weights"][t, j].double()[:, None])
        return out
    if kind == "linear":
        v = s["x"].double()
        if case["swiglu"]:
            v = v[:, :case["K"]] * torch.sigmoid(v[:, :case["K"]]) * v[:, case["K"]:]
        x = _exact_quant(v)
    else:
        x = _exact_unpack(s["xq"], s["xs"])
        x = x[s["row_token"].long()] if E else x
    if not E:
        return x @ _exact_unpack(s["wq"], s["ws"]).t()
    bounds = s["offsets"].tolist()
    y = torch.zeros(bounds[-1], case["N"], dtype=torch.float64, device="cuda")
    for e in range(E):
        if bounds[e + 1] > bounds[e]:
            y[bounds[e]:bounds[e + 1]] = x[bounds[e]:bounds[e + 1]] @ _exact_unpack(s["wq"][e], s["ws"][e]).t()
    return y
