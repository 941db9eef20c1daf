"""Cases of the expert products that work on row-major weights: the 16-bit
grouped product with its gradients, and the int8 product with one scale per
token and one per channel.

Shapes are those of the MoE layers of this repository (H=4096, E=64, top-8,
I=1536; H=7168, I=2048; the tiny H=256, E=8, I=128 layer) and generic ones
around them.  Rows come from a top-k routing of T tokens: expert popularity
falls as rank^-skew (0 is uniform), so groups are ragged and some stay empty.

Kinds of cases
  mm      y = x W_e^T over ragged groups of rows (serving and the forward pass)
  step    the same with its backward pass: y, dx and dW from dy
  linear  16-bit activations (through SwiGLU where `swiglu`) quantised to int8
          per token, times int8 weights: dense (E = 0) or grouped by expert
  mm_i8   the int8 product with the codes in hand, rows gathered from tokens
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the smallest call: a tiny layer, 37 tokens to one expert each, bound by latency
        dict(name="mm_tiny_fp16", kind="mm", T=37, topk=1, E=8, K=256, N=128, dtype="fp16", skew=0.0),
        # decoding one token through the gate projection of 8 of 64 experts: bound by the weights' bytes
        dict(name="mm_one_token_bf16", kind="mm", T=1, topk=8, E=64, K=4096, N=1536, dtype="bf16", skew=0.0),
        # a decode batch of 61 sequences through the down projection, popular experts hit more often
        dict(name="mm_decode_fp16", kind="mm", T=61, topk=8, E=64, K=1536, N=4096, dtype="fp16", skew=0.5),
        # a prompt of 4096 tokens through the gate projection: bound by the matrix units
        dict(name="mm_prefill_bf16", kind="mm", T=4096, topk=8, E=64, K=4096, N=1536, dtype="bf16", skew=0.3),
        # one training step of a layer with 16 experts on this GPU
        dict(name="step_bf16", kind="step", T=8192, topk=2, E=16, K=2048, N=4096, dtype="bf16", skew=0.3),
        # a small fine-tuning step: sizes that fill no tile, experts without a row
        dict(name="step_odd_fp16", kind="step", T=301, topk=2, E=24, K=1000, N=520, dtype="fp16", skew=1.2),
        # many small experts, about 190 rows each
        dict(name="step_many_experts_bf16", kind="step", T=1531, topk=8, E=64, K=2048, N=1408, dtype="bf16",
             skew=0.3),
        # one token through a dense int8 projection (a shared expert's): bound by the weights' bytes
        dict(name="linear_one_token_bf16", kind="linear", T=1, topk=1, E=0, K=7168, N=4096, dtype="bf16",
             swiglu=False, skew=0.0),
        # the down projection of a decode batch: SwiGLU, quantisation and the grouped product
        dict(name="linear_decode_swiglu_bf16", kind="linear", T=61, topk=8, E=64, K=1536, N=4096, dtype="bf16",
             swiglu=True, skew=0.5),
        # a prompt through a dense projection
        dict(name="linear_prefill_fp16", kind="linear", T=4099, topk=1, E=0, K=7168, N=4096, dtype="fp16",
             swiglu=False, skew=0.0),
        # a decode batch with the quantised tokens in hand, to fp32 rows
        dict(name="mm_i8_decode_fp32", kind="mm_i8", T=19, topk=8, E=128, K=4096, N=2048, dtype="fp32", skew=0.5),
        # a prompt of 4096 tokens, gathered to the experts' rows
        dict(name="mm_i8_prefill_bf16", kind="mm_i8", T=4096, topk=8, E=64, K=4096, N=1536, dtype="bf16", skew=0.3),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["mm", "step", "linear", "mm_i8"])
    step = 16 if kind in ("linear", "mm_i8") else 8  # a row is a multiple of 16 bytes
    K = _log_int(rng, 128, 7168, step)
    N = _log_int(rng, 128, 4096, 8)
    E = rng.choice([0, rng.randint(2, 64)]) if kind in ("linear", "mm_i8") else rng.randint(1, 64)
    topk = rng.randint(1, min(8, max(1, E)))
    most = 2e11 / (K * N * (3 if kind == "step" else 1))  # a drawn case costs no more than a listed one
    rows = _log_int(rng, 1, int(max(1, min(32768, most))))
    T = max(1, rows // topk)
    c = dict(kind=kind, T=T, topk=topk, E=E, K=K, N=N, skew=rng.choice([0.0, 0.5, 1.2]))
    c["dtype"] = rng.choice(["bf16", "fp16", "fp32"]) if kind == "mm_i8" else rng.choice(["bf16", "fp16"])
    if kind == "linear":
        c["swiglu"] = rng.random() < 0.5
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _popularity(case):
    E = case["E"]
    p = [(e + 1) ** -case["skew"] for e in range(E)]
    s = sum(p)
    return [v / s for v in p]


def _route(case, g):
    """offsets int32 [E + 1], the token of each row int32 [rows], and the host's view of the largest group."""
    E, T, k = case["E"], case["T"], case["topk"]
    p = torch.tensor(_popularity(case), device="cuda")
    score = p.log() - (-torch.rand(T, E, device="cuda", generator=g).clamp_min(1e-20).log()).log()
    ids = score.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offsets, (order // k).to(torch.int32), int(counts.max())


def _randn(shape, scale, dtype, g):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.reshape(-1).split(1 << 26):
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) * scale)
    return out


def _weights_i8(E, N, K, g):
    """int8 codes [E, N, K] of normal weights and one fp32 scale per output channel [E, N]."""
    codes = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    scales = torch.empty(E, N, dtype=torch.float32, device="cuda")
    for e in range(E):
        w = torch.randn(N, K, device="cuda", generator=g) * 0.02
        s = w.abs().amax(1) / 127
        codes[e] = (w / s[:, None]).round().clamp(-127, 127).to(torch.int8)
        scales[e] = s
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    T, k, E, K, N = (case[n] for n in ("T", "topk", "E", "K", "N"))
    rows, kind, dt = T * k, case["kind"], DTYPES[case["dtype"]]
    s = dict(case)
    if E:
        s["offsets"], s["row_token"], s["most"] = _route(case, g)
    if kind in ("mm", "step"):
        s["x"] = _randn((rows, K), 1.0, dt, g)
        s["w"] = _randn((E, N, K), 0.02, dt, g)
        if kind == "step":
            s["dy"] = _randn((rows, N), 0.05, dt, g)
            s["x"].requires_grad_()
            s["w"].requires_grad_()
        return s
    s["wq"], s["ws"] = _weights_i8(max(1, E), N, K, g)
    if not E:
        s["wq"], s["ws"] = s["wq"][0], s["ws"][0]
    if kind == "linear":
        # tokens differ in size, as rows of a residual stream do
        size = torch.exp(torch.randn(rows, 1, device="cuda", generator=g) * 0.5)
        width = 2 * K if case["swiglu"] else K
        s["x"] = (torch.randn(rows, width, device="cuda", generator=g) * size).to(dt)
    else:
        x = torch.randn(T, K, device="cuda", generator=g)
        s["xs"] = x.abs().amax(1) / 127
        s["xq"] = (x / s["xs"][:, None]).round().clamp(-127, 127).to(torch.int8)
        if not E:
            s["row_token"] = None
    return s


# ------------------------------------------------------------------ plain forms
def _slots(offsets, most, rows):
    """Place of each row in a [E, most] grid of rows: the groups padded to the largest one."""
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].contiguous(), r.to(offsets.dtype), right=True)
    return e * most + (r - offsets[e])


def _padded(v, slots, E, most):
    out = torch.zeros(E * most, v.shape[1], dtype=torch.float32, device=v.device)
    out[slots] = v.float()
    return out.view(E, most, v.shape[1])


def _grouped(x, w, slots, most):
    """fp32 x[r] @ w[e]^T for the rows r of each group e."""
    E, N, _ = w.shape
    xt = _padded(x, slots, E, most).transpose(1, 2).contiguous()
    return torch.bmm(w.float(), xt).transpose(1, 2).reshape(E * most, N)[slots]


def _plain_mm(s):
    x, w = s["x"].detach(), s["w"].detach()
    slots = _slots(s["offsets"], s["most"], x.shape[0])
    return _grouped(x, w, slots, s["most"]).to(x.dtype)


def _plain_step(s):
    x, w, dy, most = s["x"].detach(), s["w"].detach(), s["dy"], s["most"]
    E, N, K = w.shape
    slots = _slots(s["offsets"], most, x.shape[0])
    y = _grouped(x, w, slots, most)
    xp, dyp = _padded(x, slots, E, most), _padded(dy, slots, E, most)
    dx = torch.bmm(dyp, w.float()).view(E * most, K)[slots]
    dw = torch.bmm(dyp.transpose(1, 2).contiguous(), xp)
    return y.to(x.dtype), dx.to(x.dtype), dw.to(x.dtype)


def _plain_quant(x, swiglu):
    v = x.float()
    if swiglu:
        gate, up = v.chunk(2, dim=1)
        v = gate / (1 + torch.exp(-gate)) * up
    # one division, rounded once (a Python number over a tensor is a reciprocal and a product)
    mult = v.new_full((), 127.0) / v.abs().amax(1).clamp_min(2.0 ** -64)
    return torch.round(v * mult[:, None]), mult.reciprocal()


def _plain_mm_i8(s, codes, scale):
    """codes [rows, K] and scale [rows] in fp32."""
    if s["E"]:
        slots = _slots(s["offsets"], s["most"], codes.shape[0])
        acc = _grouped(codes, s["wq"], slots, s["most"])
        e = torch.div(slots, s["most"], rounding_mode="floor")
        return acc * scale[:, None] * s["ws"][e]
    return codes @ s["wq"].float().t() * scale[:, None] * s["ws"]


def _plain(s):
    kind = s["kind"]
    if kind == "mm":
        return _plain_mm(s)
    if kind == "step":
        return _plain_step(s)
    if kind == "linear":
        return _plain_mm_i8(s, *_plain_quant(s["x"], s["swiglu"])).to(s["x"].dtype)
    codes, scale = s["xq"].float(), s["xs"]
    if s["E"]:
        t = s["row_token"].long()
        codes, scale = codes[t], scale[t]
    return _plain_mm_i8(s, codes, scale).to(DTYPES[s["dtype"]])


def run(state):
    if not own:
        return _plain(state)
    import bit_grouped_gemm_amd as moe
    kind, offsets = state["kind"], state.get("offsets")
    if kind == "mm":
        return moe.moe_grouped_mm(state["x"], state["w"], offsets)
    if kind == "step":
        y = moe.moe_grouped_mm(state["x"], state["w"], offsets)
        dx, dw = torch.autograd.grad(y, (state["x"], state["w"]), state["dy"])
        return y, dx, dw
    if kind == "linear":
        return moe.moe_linear_i8(state["x"], state["wq"], state["ws"], offsets, swiglu=state["swiglu"])
    return moe.moe_mm_i8(state["xq"], state["xs"], state["wq"], state["ws"], offsets, row_token=state["row_token"],
                         out_dtype=DTYPES[state["dtype"]])


def work(case):
    T, k, E, K, N = (case[n] for n in ("T", "topk", "E", "K", "N"))
    rows, kind = T * k, case["kind"]
    # experts that get a row, each slot taken as a draw from the popularity
    touched = sum(1 - (1 - min(1.0, k * p)) ** T for p in _popularity(case)) if E else 1
    touched = min(touched, rows)
    flops = 2.0 * rows * K * N
    if kind == "mm":
        return {"bytes": 2.0 * (rows * (K + N) + touched * K * N), "flops": flops}
    if kind == "step":
        # x, dy and the touched weights in; y, dx and every expert's gradient out
        return {"bytes": 2.0 * (2 * rows * (K + N) + (touched + E) * K * N), "flops": 3 * flops}
    if kind == "linear":
        wide = 2 if case["swiglu"] else 1
        return {"bytes": 2.0 * rows * (wide * K + N) + touched * (K * N + 4.0 * N), "flops": flops}
    out = 4.0 if case["dtype"] == "fp32" else 2.0
    tokens = T if E else rows
    return {"bytes": tokens * (K + 4.0) + out * rows * N + touched * (K * N + 4.0 * N), "flops": flops}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind, E = case["kind"], case["E"]
    bounds = s["offsets"].tolist() if E else [0, case["T"] * case["topk"]]
    w = (s["w"] if kind in ("mm", "step") else s["wq"]).detach()
    w = w if E else w[None]
    rows, N, K = bounds[-1], w.shape[1], w.shape[2]

    if kind in ("mm", "step"):
        x, scale, ws = s["x"].detach().double(), None, None
    else:
        ws = (s["ws"] if E else s["ws"][None]).double()
        if kind == "linear":
            x = s["x"].double()
            if case["swiglu"]:
                x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
            top = x.abs().amax(dim=1, keepdim=True).clamp_min(2.0 ** -64)
            x, scale = torch.round(x * 127 / top), top / 127
        else:
            x, scale = s["xq"].double(), s["xs"].double()[:, None]
            if E:
                x, scale = x[s["row_token"].long()], scale[s["row_token"].long()]

    y = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    if kind == "step":
        dx = torch.zeros(rows, K, dtype=torch.float64, device="cuda")
        dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for e in range(w.shape[0]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        we = w[e].double()
        y[a:b] = x[a:b] @ we.t()
        if scale is not None:
            y[a:b] *= scale[a:b] * ws[e]
        if kind == "step":
            d = s["dy"][a:b].double()
            dx[a:b] = d @ we
            dw[e] = d.t() @ x[a:b]
    return (y, dx, dw) if kind == "step" else y
