"""Python binding of the MI355X low-bit MoE expert layer (libmoe.so).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI in ``include/moe.h``.  PyTorch provides device memory and
the current stream.  There is no CPU or PyTorch fallback: if the library is
missing, importing the entry points raises.

Entry points (same names as the C ABI):
    moe_workspace_size(cfg) -> int
    moe_permute(cfg, x, topk_ids, ws=None) -> (counts, offsets, expand_idx, row_token, xq, xs)
    moe_grouped_gemm1_swiglu(cfg, xq, xs, row_token, offsets, weights, ws) -> (hq, hs)
    moe_grouped_gemm2(cfg, hq, hs, offsets, weights, ws) -> y
    moe_combine(cfg, y, expand_idx, offsets, topk_weights) -> out
    moe_layer(cfg, x, topk_ids, topk_weights, weights, ws=None, out=None) -> out
    moe_layer_static(cfg, x, topk_ids, topk_weights, weights, out=None) -> out   (no workspace)
    moe_layer_persistent(cfg, x, topk_ids, topk_weights, weights, ws=None, out=None, status=None) -> out
                                                                   (decode shapes: one launch)
    moe_prepack_weights(cfg, weights) -> TiledWeights
    moe_route(cfg, x, gate_w) -> (topk_ids, topk_weights)   (the router in front of the layer)
    moe_encode_e4m3(v) -> codes   (diagnostic: the quantisers' fp32 -> e4m3 conversion)
and on row-major weights (nothing to prepack):
    moe_grouped_mm(x, w, offsets) -> y   (bf16 / fp16 experts; differentiable)
    moe_grouped_mm_dgrad(dy, w, offsets) -> dx,  moe_grouped_mm_wgrad(dy, x, offsets) -> dw
    moe_quant_i8(x, swiglu=False) -> (codes, scales)   (int8, one scale per token)
    moe_mm_i8(xq, xs, wq, ws, offsets=None, row_token=None) -> y   (grouped or dense)
    moe_linear_i8(x, wq, ws, offsets=None, row_token=None, swiglu=False) -> y   (both in one call)

The layer's GEMM entry points read expert weights in the tiled layout: convert the
canonical row-major tensors once with moe_prepack_weights(cfg, weights)
(a one-time step at weight load).
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import os
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libmoe.so")

MOE_OK = 0
MOE_ERR_NULL_ARG = 1
MOE_ERR_BAD_SHAPE = 2
MOE_ERR_UNSUPPORTED = 3
MOE_ERR_WORKSPACE = 4
MOE_ERR_MISALIGNED = 5
MOE_ERR_HIP = 6

WFMT_FP8_BLOCK = 0
WFMT_MXFP4 = 1
WFMT_NVFP4 = 2
RATE_E2M1_E2M1 = 16  # moe_mfma_rate's e2m1 x e2m1 operand pair

EXPORTS = ("moe_workspace_size", "moe_permute", "moe_grouped_gemm1_swiglu", "moe_grouped_gemm2",
           "moe_combine", "moe_layer", "moe_layer_static", "moe_layer_persistent", "moe_layer_persistent_spin_limit",
           "moe_prepack_weights",
           "moe_stream_read",
           "moe_mfma_rate", "moe_encode_e4m3", "moe_route", "moe_route_workspace_size", "moe_status_str",
           "moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad",
           "moe_grouped_mm_wgrad_workspace_size", "moe_quant_i8", "moe_mm_i8",
           "moe_linear_i8", "moe_linear_i8_workspace_size")

# element types of the row-major products
_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class MoeCfg(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("T", "H", "I", "E", "topk", "wfmt", "wblk", "act_group",
                                          "has_shared", "act_fmt")]


class MoeWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("w1", "w1s", "w2", "w2s", "sw1", "sw1s", "sw2", "sw2s")] + \
        [("prepacked", C.c_int32)] + [(n, C.c_void_p) for n in ("w1g", "w2g", "sw1g", "sw2g")]


class MoeMmCfg(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("R", "N", "K", "E", "T", "dtype", "out_dtype", "clear_rest")]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({status_str(status)})")


_lib: Optional[C.CDLL] = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with bit_grouped_gemm_amd.build.build() "
                          "(hipcc, gfx950); there is no fallback implementation")
    L = C.CDLL(path)
    vp, sz = C.c_void_p, C.c_size_t
    cfgp = C.POINTER(MoeCfg)
    wp = C.POINTER(MoeWeights)
    L.moe_workspace_size.argtypes = [cfgp, C.POINTER(sz)]
    L.moe_permute.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_grouped_gemm1_swiglu.argtypes = [cfgp, vp, vp, vp, vp, wp, vp, vp, vp, sz, vp]
    L.moe_grouped_gemm2.argtypes = [cfgp, vp, vp, vp, wp, vp, vp, sz, vp]
    L.moe_combine.argtypes = [cfgp, vp, vp, vp, vp, vp, vp]
    L.moe_layer.argtypes = [cfgp, vp, vp, vp, wp, vp, vp, sz, vp]
    L.moe_layer_static.argtypes = [cfgp, vp, vp, vp, wp, vp, vp]
    L.moe_layer_persistent.argtypes = [cfgp, vp, vp, vp, wp, vp, vp, sz, vp, vp]
    L.moe_layer_persistent_spin_limit.argtypes = [C.c_int]
    L.moe_prepack_weights.argtypes = [cfgp, wp, wp, vp]
    L.moe_stream_read.argtypes = [vp, sz, vp, sz, vp]
    L.moe_mfma_rate.argtypes = [C.c_int, C.c_int, vp, sz, C.POINTER(C.c_double), vp]
    L.moe_encode_e4m3.argtypes = [vp, sz, vp, vp]
    L.moe_route_workspace_size.argtypes = [cfgp, C.POINTER(sz)]
    L.moe_route.argtypes = [cfgp, vp, vp, vp, vp, vp, sz, vp]
    mmp = C.POINTER(MoeMmCfg)
    L.moe_grouped_mm.argtypes = [mmp, vp, vp, vp, vp, vp]
    L.moe_grouped_mm_dgrad.argtypes = [mmp, vp, vp, vp, vp, vp]
    L.moe_grouped_mm_wgrad.argtypes = [mmp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_grouped_mm_wgrad_workspace_size.argtypes = [mmp, C.POINTER(sz)]
    L.moe_quant_i8.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp, vp]
    L.moe_mm_i8.argtypes = [mmp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_linear_i8_workspace_size.argtypes = [mmp, C.c_int, C.POINTER(sz)]
    L.moe_linear_i8.argtypes = [mmp, vp, C.c_int, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_status_str.argtypes = [C.c_int]
    L.moe_status_str.restype = C.c_char_p
    for n in EXPORTS:
        if n != "moe_status_str":
            getattr(L, n).restype = C.c_int
    _lib = L
    return L


def status_str(status: int) -> str:
    return load().moe_status_str(int(status)).decode()


# ------------------------------------------------------------------ helpers
@dataclasses.dataclass(frozen=True)
class Cfg:
    T: int
    H: int
    I: int
    E: int
    topk: int
    wfmt: int
    wblk: int
    act_group: int
    has_shared: int = 0
    act_fmt: int = 0  # 0: e4m3 + fp32 scale per act_group; 1: MXFP4 (e2m1 + e8m0 per 32)

    def c(self) -> MoeCfg:
        return MoeCfg(self.T, self.H, self.I, self.E, self.topk, self.wfmt, self.wblk, self.act_group,
                      self.has_shared, self.act_fmt)

    @classmethod
    def for_workload(cls, wl, T: int) -> "Cfg":
        return cls(T, wl.H, wl.I, wl.E, wl.topk, wl.wfmt, wl.wblk, wl.act_group, int(wl.shared),
                   int(getattr(wl, "act_fmt", 0)))

    def act_tensors(self, rows: int, width: int, device) -> Tuple[torch.Tensor, torch.Tensor]:
        """Empty (codes, scales) of `rows` quantised activation rows of `width`
        channels: e4m3 [rows][width] + fp32 [rows][width / act_group], or for
        MXFP4 e2m1 pairs [rows][width / 2] + e8m0 [rows][width / 32]."""
        if self.act_fmt == 1:
            return (torch.empty(rows, width // 2, dtype=torch.uint8, device=device),
                    torch.empty(rows, width // 32, dtype=torch.uint8, device=device))
        return (torch.empty(rows, width, dtype=torch.uint8, device=device),
                torch.empty(rows, width // self.act_group, dtype=torch.float32, device=device))

    def with_T(self, T: int) -> "Cfg":
        return dataclasses.replace(self, T=T)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the HIP library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the HIP library must be contiguous")
    return t.data_ptr() or None


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _check(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def weights_struct(w) -> MoeWeights:
    """moe_weights from an object with w1, w1s, w2, w2s[, sw1, sw1s, sw2, sw2s] tensors,
    NVFP4's matrix scales w1g, w2g[, sw1g, sw2g] and an optional `prepacked` flag
    (absent: 0, the canonical row-major layout)."""
    g = lambda n: _ptr(getattr(w, n, None))
    return MoeWeights(g("w1"), g("w1s"), g("w2"), g("w2s"), g("sw1"), g("sw1s"), g("sw2"), g("sw2s"),
                      int(getattr(w, "prepacked", 0)), g("w1g"), g("w2g"), g("sw1g"), g("sw2g"))


def _u16(x: torch.Tensor) -> torch.Tensor:
    return x.view(torch.int16) if x.dtype == torch.bfloat16 else x


# ------------------------------------------------------------------ entry points
def moe_workspace_size(cfg: Cfg) -> int:
    n = C.c_size_t(0)
    c = cfg.c()
    _check("moe_workspace_size", load().moe_workspace_size(C.byref(c), C.byref(n)))
    return int(n.value)


def workspace(cfg: Cfg, device="cuda") -> torch.Tensor:
    return torch.empty(moe_workspace_size(cfg), dtype=torch.uint8, device=device)


def moe_permute(cfg: Cfg, x: torch.Tensor, topk_ids: torch.Tensor, ws: Optional[torch.Tensor] = None):
    dev = x.device
    T, k, E, sh = cfg.T, cfg.topk, cfg.E, cfg.has_shared
    counts = torch.empty(E + sh, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1 + sh, dtype=torch.int32, device=dev)
    eidx = torch.empty(T * k, dtype=torch.int32, device=dev)
    rtok = torch.empty(T * k + T * sh, dtype=torch.int32, device=dev)
    xq, xs = cfg.act_tensors(T, cfg.H, dev)
    c = cfg.c()
    ws = workspace(cfg, dev) if ws is None else ws  # per-chunk counts when T*topk > 4096
    _check("moe_permute", load().moe_permute(C.byref(c), _ptr(_u16(x)), _ptr(topk_ids), _ptr(counts),
                                             _ptr(offsets), _ptr(eidx), _ptr(rtok), _ptr(xq), _ptr(xs),
                                             _ptr(ws), ws.numel(), _stream()))
    return counts, offsets, eidx, rtok, xq, xs


def moe_grouped_gemm1_swiglu(cfg: Cfg, xq, xs, row_token, offsets, weights, ws: Optional[torch.Tensor] = None,
                             rows: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    dev = xq.device
    R = rows if rows is not None else cfg.T * cfg.topk + cfg.T * cfg.has_shared
    hq, hs = cfg.act_tensors(R, cfg.I, dev)
    ws = workspace(cfg, dev) if ws is None else ws
    c, w = cfg.c(), weights_struct(weights)
    _check("moe_grouped_gemm1_swiglu",
           load().moe_grouped_gemm1_swiglu(C.byref(c), _ptr(xq), _ptr(xs), _ptr(row_token), _ptr(offsets),
                                           C.byref(w), _ptr(hq), _ptr(hs), _ptr(ws), ws.numel(), _stream()))
    return hq, hs


def moe_grouped_gemm2(cfg: Cfg, hq, hs, offsets, weights, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    dev = hq.device
    y = torch.empty(hq.shape[0], cfg.H, dtype=torch.float32, device=dev)
    ws = workspace(cfg, dev) if ws is None else ws
    c, w = cfg.c(), weights_struct(weights)
    _check("moe_grouped_gemm2",
           load().moe_grouped_gemm2(C.byref(c), _ptr(hq), _ptr(hs), _ptr(offsets), C.byref(w), _ptr(y),
                                    _ptr(ws), ws.numel(), _stream()))
    return y


def moe_combine(cfg: Cfg, y, expand_idx, offsets, topk_weights) -> torch.Tensor:
    out = torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=y.device)
    c = cfg.c()
    _check("moe_combine", load().moe_combine(C.byref(c), _ptr(y), _ptr(expand_idx), _ptr(offsets),
                                             _ptr(topk_weights), _ptr(_u16(out)), _stream()))
    return out


def moe_layer(cfg: Cfg, x, topk_ids, topk_weights, weights, ws: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    if out is None:
        out = torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=x.device)
    ws = workspace(cfg, x.device) if ws is None else ws
    c, w = cfg.c(), weights_struct(weights)
    _check("moe_layer", load().moe_layer(C.byref(c), _ptr(_u16(x)), _ptr(topk_ids), _ptr(topk_weights), C.byref(w),
                                         _ptr(_u16(out)), _ptr(ws), ws.numel(), _stream()))
    return out


STATIC_SCRATCH_BYTES = 64 << 20  # MOE_STATIC_SCRATCH_BYTES


def moe_layer_static(cfg: Cfg, x, topk_ids, topk_weights, weights,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_layer with the library's static per-GPU scratch instead of a
    workspace (the call allocates nothing on the library side)."""
    if out is None:
        out = torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=x.device)
    c, w = cfg.c(), weights_struct(weights)
    _check("moe_layer_static", load().moe_layer_static(C.byref(c), _ptr(_u16(x)), _ptr(topk_ids), _ptr(topk_weights),
                                                       C.byref(w), _ptr(_u16(out)), _stream()))
    return out


def moe_layer_persistent(cfg: Cfg, x, topk_ids, topk_weights, weights, ws: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_layer as one persistent launch (decode shapes; raises with
    MOE_ERR_UNSUPPORTED otherwise).  `status`, an int32 device tensor of one
    element, receives the number of expired waits (0 in a correct run)."""
    if out is None:
        out = torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=x.device)
    ws = workspace(cfg, x.device) if ws is None else ws
    c, w = cfg.c(), weights_struct(weights)
    _check("moe_layer_persistent",
           load().moe_layer_persistent(C.byref(c), _ptr(_u16(x)), _ptr(topk_ids), _ptr(topk_weights), C.byref(w),
                                       _ptr(_u16(out)), _ptr(ws), ws.numel(), _ptr(status), _stream()))
    return out


PERSIST_SPIN_LIMIT = 1 << 20  # moe_layer_persistent's default polls per wait


def moe_layer_persistent_spin_limit(polls: int) -> None:
    """Polls per wait of moe_layer_persistent before it expires (process-wide;
    0 exercises the expiry path)."""
    _check("moe_layer_persistent_spin_limit", load().moe_layer_persistent_spin_limit(int(polls)))


@dataclasses.dataclass
class TiledWeights:
    """Expert weights in the layout the GEMM entry points read (prepacked = 1)."""
    w1: torch.Tensor
    w1s: torch.Tensor
    w2: torch.Tensor
    w2s: torch.Tensor
    sw1: Optional[torch.Tensor] = None
    sw1s: Optional[torch.Tensor] = None
    sw2: Optional[torch.Tensor] = None
    sw2s: Optional[torch.Tensor] = None
    prepacked: int = 1
    w1g: Optional[torch.Tensor] = None   # NVFP4: fp32 matrix scales (row-major, unchanged)
    w2g: Optional[torch.Tensor] = None
    sw1g: Optional[torch.Tensor] = None
    sw2g: Optional[torch.Tensor] = None


def moe_prepack_weights(cfg: Cfg, weights) -> TiledWeights:
    """Tiled copies of a layer's canonical row-major weights (w1, w1s, w2, w2s
    and, when cfg.has_shared, sw1..sw2s): the one-time step at weight load."""
    names = ["w1", "w1s", "w2", "w2s"] + (["sw1", "sw1s", "sw2", "sw2s"] if cfg.has_shared else [])
    if cfg.wfmt == WFMT_NVFP4:
        names += ["w1g", "w2g"] + (["sw1g", "sw2g"] if cfg.has_shared else [])
    out = TiledWeights(**{n: torch.empty_like(getattr(weights, n)) for n in names})
    c, src, dst = cfg.c(), weights_struct(weights), weights_struct(out)
    dst.prepacked = 0
    _check("moe_prepack_weights", load().moe_prepack_weights(C.byref(c), C.byref(src), C.byref(dst), _stream()))
    out.prepacked = int(dst.prepacked)
    return out





def moe_stream_read(buf: torch.Tensor, sink: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Read every byte of a device buffer once (a plain HBM read stream);
    returns the sink (one folded word per workgroup, one workgroup per CU)."""
    if sink is None:
        sink = torch.empty(8192, dtype=torch.int32, device=buf.device)
    _check("moe_stream_read", load().moe_stream_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                                      sink.numel() * sink.element_size(), _stream()))
    return sink


def moe_mfma_rate(wfmt: int, iters: int, sink: torch.Tensor) -> float:
    """Enqueue the scaled-MFMA rate probe (all operands 1.0); returns the FLOP
    count enqueued.  `sink` (float32, device) receives 4096 * iters per
    workgroup."""
    flops = C.c_double(0.0)
    _check("moe_mfma_rate", load().moe_mfma_rate(int(wfmt), int(iters), _ptr(sink),
                                                  sink.numel() * sink.element_size(), C.byref(flops), _stream()))
    return flops.value


def moe_route_workspace_size(cfg: Cfg) -> int:
    n = C.c_size_t(0)
    c = cfg.c()
    _check("moe_route_workspace_size", load().moe_route_workspace_size(C.byref(c), C.byref(n)))
    return int(n.value)


def moe_route(cfg: Cfg, x: torch.Tensor, gate_w: torch.Tensor, ids: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Router: bf16 x [T,H] and gate rows [E,H] -> (topk_ids int32 [T,topk],
    topk_weights fp32 [T,topk]), the layer's routing inputs."""
    if ids is None:
        ids = torch.empty(cfg.T, cfg.topk, dtype=torch.int32, device=x.device)
    if weights is None:
        weights = torch.empty(cfg.T, cfg.topk, dtype=torch.float32, device=x.device)
    if ws is None:
        n = moe_route_workspace_size(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    c = cfg.c()
    _check("moe_route", load().moe_route(C.byref(c), _ptr(_u16(x)), _ptr(_u16(gate_w)), _ptr(ids), _ptr(weights),
                                         _ptr(ws), 0 if ws is None else ws.numel(), _stream()))
    return ids, weights


def moe_encode_e4m3(v: torch.Tensor, codes: Optional[torch.Tensor] = None) -> torch.Tensor:
    """e4m3 codes (uint8, same shape) of fp32 values by the quantisers' conversion."""
    if codes is None:
        codes = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check("moe_encode_e4m3", load().moe_encode_e4m3(_ptr(v), v.numel(), _ptr(codes), _stream()))
    return codes


# ------------------------------------------------------------------ row-major products
_16BIT = (torch.bfloat16, torch.float16)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


def _call(name: str, index: int, *args) -> None:
    """A library call on the current stream of device `index`, with that device current."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            rc = getattr(_lib or load(), name)(*args, _raw_stream(index))
    else:
        rc = getattr(_lib or load(), name)(*args, _raw_stream(index))
    if rc:
        raise MoeError(name, rc)


def _addr(name: str, t: torch.Tensor, dtypes, shape, dev: torch.device):
    """The address of a contiguous GPU tensor of one of `dtypes`, of `shape`
    (None: any size) and on `dev`; None where it is empty.  A message is only
    put together for a tensor that is none."""
    if t.dtype in dtypes and t.shape == shape and t.device == dev and t.is_cuda and t.is_contiguous():
        return t.data_ptr() or None
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of {', '.join(map(str, dtypes))}")
    if t.dim() != len(shape) or any(w is not None and h != w for h, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple('any' if v is None else v for v in shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")
    return _ptr(t)


_grad_enabled = torch.is_grad_enabled


def _refuse_derivatives(name: str, out: Optional[torch.Tensor], a: Optional[torch.Tensor] = None,
                        b: Optional[torch.Tensor] = None) -> None:
    """Refuses operands (and outputs) that need a gradient or carry a forward-mode
    tangent, of which the result would be cut off without a word."""
    if _grad_enabled() and (a is not None and a.requires_grad or b is not None and b.requires_grad
                            or out is not None and out.requires_grad):
        raise ValueError(f"{name} has no gradient: call it under torch.no_grad() or detach its operands")
    if forward_ad._current_level >= 0:  # in a dual level
        _refuse_tangents(name, out, a, b)


def _refuse_tangents(name: str, *tensors: Optional[torch.Tensor]) -> None:
    """The same for tangents alone: a dual tensor does not say that it needs a
    gradient, and torch.no_grad() leaves forward mode on."""
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError(f"{name} has no forward-mode derivative: give it operands without a tangent")


def _new_or_checked(out, shape, dtype, allowed, like):
    """The output tensor and clear_rest: a new one has every row written, a
    caller's keeps its rows of no group."""
    if out is not None:
        return out, 0
    if dtype not in allowed:
        raise ValueError(f"out_dtype {dtype} is not one of {', '.join(map(str, allowed))}")
    return like.new_empty(shape, dtype=dtype), 1


# Tells autograd that a call wrote into a caller's tensor, so that a backward pass
# which saved it raises instead of using the new values.
_written = torch.autograd.graph.increment_version


def _matrices(w: torch.Tensor):
    if w.dim() != 3:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected (E, N, K)")
    if max(w.shape) > 0x7FFFFFFF:
        raise ValueError(f"w: shape {tuple(w.shape)}, sizes are at most 2^31 - 1")
    return w.shape


def _rows_of(name: str, t: torch.Tensor) -> torch.Size:
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected two dimensions")
    if t.shape[0] > 0x7FFFFFFF:
        raise ValueError(f"{name}: {t.shape[0]} rows, at most 2^31 - 1")
    return t.shape


def _grouped(name, rows, p, w, offsets, width, other, out, out_dtype):
    """y from x, or dx from dy: `p` [R, width] times the matrices w [E, N, K]."""
    R, dt, dev = _rows_of(rows, p)[0], p.dtype, p.device
    E, N, K = w.shape
    allowed = (dt, torch.float32)
    pp = _addr(rows, p, _16BIT, (R, width), dev)
    pw = _addr("w", w, (dt,), (E, N, K), dev)
    po = _addr("offsets", offsets, (torch.int32,), (E + 1,), dev)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    given = out
    out, clear = _new_or_checked(out, (R, other), out_dtype or dt, allowed, p)
    py = _addr("out", out, allowed, (R, other), dev)
    c = MoeMmCfg(R, N, K, E, 0, _DT[dt], _DT[out.dtype], clear)
    _call(name, dev.index, C.byref(c), pp, pw, po, py)
    if given is not None:
        _written(given)
    return out


def _grouped_mm(x, w, offsets, out=None, out_dtype=None):
    _, N, K = _matrices(w)
    return _grouped("moe_grouped_mm", "x", x, w, offsets, K, N, out, out_dtype)


def moe_grouped_mm_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                         out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """dx [R, K] = dy[r] @ w[e] for the rows r of each group e: moe_grouped_mm's
    gradient with respect to x.  `out` and `out_dtype` as in moe_grouped_mm.
    Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_grouped_mm_dgrad", out, dy, w)
    _, N, K = _matrices(w)
    return _grouped("moe_grouped_mm_dgrad", "dy", dy, w, offsets, N, K, out, out_dtype)


def moe_grouped_mm_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                         out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                         work: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dw [E, N, K] = dy[r]^T x[r] summed over the rows r of each group e (zeros
    for an empty group): moe_grouped_mm's gradient with respect to w.
    `out_dtype`: dy's (default) or torch.float32; `out` is fully overwritten.
    `work`: uint8 scratch of at least moe_grouped_mm_wgrad_workspace_size(...)
    bytes, allocated where absent and needed.  Not differentiable: operands that
    need a gradient are refused."""
    _refuse_derivatives("moe_grouped_mm_wgrad", out, dy, x)
    (R, N), K, dt, dev = _rows_of("dy", dy), _rows_of("x", x)[1], dy.dtype, dy.device
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected (E + 1,)")
    E = offsets.shape[0] - 1
    allowed = (dt, torch.float32)
    pd = _addr("dy", dy, _16BIT, (R, N), dev)
    px = _addr("x", x, (dt,), (R, K), dev)
    po = _addr("offsets", offsets, (torch.int32,), (E + 1,), dev)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    given = out
    out, _ = _new_or_checked(out, (E, N, K), out_dtype or dt, allowed, x)
    pw = _addr("out", out, allowed, (E, N, K), dev)
    c = MoeMmCfg(R, N, K, E, 0, _DT[dt], _DT[out.dtype], 0)
    if work is None:
        need = _wgrad_bytes(c)
        work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    pk = None if work is None else _addr("work", work, (torch.uint8,), work.shape, dev)
    _call("moe_grouped_mm_wgrad", dev.index, C.byref(c), pd, px, po, pw, pk, 0 if work is None else work.numel())
    if given is not None:
        _written(given)
    return out


def _wgrad_bytes(c: MoeMmCfg) -> int:
    n = C.c_size_t(0)
    _check("moe_grouped_mm_wgrad_workspace_size",
           (_lib or load()).moe_grouped_mm_wgrad_workspace_size(C.byref(c), C.byref(n)))
    return n.value


def moe_grouped_mm_wgrad_workspace_size(R: int, N: int, K: int, E: int) -> int:
    """Bytes of scratch moe_grouped_mm_wgrad needs for dy [R, N], x [R, K] and E groups."""
    return _wgrad_bytes(MoeMmCfg(R, N, K, E, 0, 0, 0, 0))


class _GroupedMM(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return _grouped_mm(x, w, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        # moe_grouped_mm_dgrad and moe_grouped_mm_wgrad, with one round of checks
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16:  # a view into something else
            dy = dy.clone()
        (E, N, K), R, dt, dev = w.shape, x.shape[0], x.dtype, x.device
        pd = _addr("dy", dy, (dt,), (R, N), dev)
        px = _addr("x", x, (dt,), (R, K), dev)
        pw = _addr("w", w, (dt,), (E, N, K), dev)
        po = _addr("offsets", offsets, (torch.int32,), (E + 1,), dev)
        c = MoeMmCfg(R, N, K, E, 0, _DT[dt], _DT[dt], 1)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = x.new_empty(x.shape)
            _call("moe_grouped_mm_dgrad", dev.index, C.byref(c), pd, pw, po, dx.data_ptr() or None)
        if ctx.needs_input_grad[1]:
            dw = w.new_empty(w.shape)
            need = _wgrad_bytes(c)
            work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            _call("moe_grouped_mm_wgrad", dev.index, C.byref(c), pd, px, po, dw.data_ptr(),
                  None if work is None else work.data_ptr(), need)
        return dx, dw, None


def moe_grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y [R, N] = x[r] @ w[e]^T for the rows r = offsets[e] .. offsets[e + 1] - 1
    of each group e, w [E, N, K] row-major.

    x and w are both bfloat16 or both float16; offsets is int32 [E + 1] on the
    same device (moe_permute's).  The result has x's type, or float32 with
    out_dtype=torch.float32 (the rows moe_combine takes).  Rows of no group (r <
    offsets[0] or r >= offsets[E]) are zeros in a new result; a caller's `out`
    keeps what it holds there.  All tensors are contiguous and on one GPU.

    Differentiable with respect to x and w (once; not with `out` or
    `out_dtype`): the gradients are moe_grouped_mm_dgrad and
    moe_grouped_mm_wgrad, and rows of no group get the gradient 0.  In a graph,
    capture forward and backward together, while no earlier result computed from
    the same leaves is kept: PyTorch ties a leaf's gradient to the stream of its first use.
    Operands with a forward-mode tangent are refused."""
    if forward_ad._current_level >= 0:
        _refuse_tangents("moe_grouped_mm", x, w, out)
    if (x.requires_grad or w.requires_grad) and _grad_enabled():
        if out is not None or out_dtype not in (None, x.dtype):
            raise ValueError("moe_grouped_mm: out and out_dtype cannot be given where a gradient is needed")
        return _GroupedMM.apply(x, w, offsets)
    if out is not None:
        _refuse_derivatives("moe_grouped_mm with out", out)
    return _grouped_mm(x, w, offsets, out, out_dtype)


def moe_quant_i8(x: torch.Tensor, swiglu: bool = False, codes: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """int8 codes [R, K] and fp32 scales [R] of the rows of x [R, K] (bfloat16 or
    float16), or of silu(gate) * up with x [R, 2 K] = gate | up where `swiglu`.
    value = code * scale; a row with an infinity or NaN gets the scale NaN.
    Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_quant_i8", scales, x)
    (R, width), dev = _rows_of("x", x), x.device
    if swiglu and width % 2:
        raise ValueError(f"x: {width} columns do not split into gate and up")
    K = width // 2 if swiglu else width
    px = _addr("x", x, _16BIT, (R, width), dev)
    given = codes, scales
    if codes is None:
        codes = torch.empty(R, K, dtype=torch.int8, device=dev)
    if scales is None:
        scales = torch.empty(R, dtype=torch.float32, device=dev)
    pq = _addr("codes", codes, (torch.int8,), (R, K), dev)
    ps = _addr("scales", scales, (torch.float32,), (R,), dev)
    _call("moe_quant_i8", dev.index, R, K, _DT[x.dtype], int(bool(swiglu)), px, pq, ps)
    for t in given:
        if t is not None:
            _written(t)
    return codes, scales


def _i8_weights(wq, ws, offsets, dev):
    """E, N, K and the addresses of int8 weights [E, N, K], or [N, K] (dense: no
    offsets), of their scales and of the offsets."""
    if wq.dim() != (2 if offsets is None else 3):
        raise ValueError(f"wq: [N, K] without offsets, [E, N, K] with offsets; got {tuple(wq.shape)}")
    E, N, K = (1, *wq.shape) if offsets is None else wq.shape
    if max(wq.shape) > 0x7FFFFFFF:
        raise ValueError(f"wq: shape {tuple(wq.shape)}, sizes are at most 2^31 - 1")
    pw = _addr("wq", wq, (torch.int8,), wq.shape, dev)
    ps = _addr("ws", ws, (torch.float32,), wq.shape[:-1], dev)
    po = None if offsets is None else _addr("offsets", offsets, (torch.int32,), (E + 1,), dev)
    return E, N, K, pw, ps, po


def _row_token(row_token, T, dev):
    if row_token is None:
        return T, None
    if row_token.dim() != 1:
        raise ValueError(f"row_token: shape {tuple(row_token.shape)}, expected one dimension")
    if row_token.shape[0] > 0x7FFFFFFF:
        raise ValueError(f"row_token: {row_token.shape[0]} rows, at most 2^31 - 1")
    return row_token.shape[0], _addr("row_token", row_token, (torch.int32,), row_token.shape, dev)


def moe_mm_i8(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
              offsets: Optional[torch.Tensor] = None, row_token: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y[r] = (xq[t] @ wq[e]^T) * xs[t] * ws[e] with int8 operands, exact integer
    sums, one scale per row of xq and one per output channel.

    Dense: wq [N, K], ws [N], every row of xq.  Grouped: wq [E, N, K], ws
    [E, N] and offsets int32 [E + 1]; with row_token int32 [R] (moe_permute's)
    row r of the result takes row t = row_token[r] of xq, else t = r.
    The result [R, N] is bfloat16 (default), float16 or float32; rows of no
    group are zeros in a new result and stay as they are in a caller's `out`.
    Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_mm_i8", out, xs, ws)
    (T, width), dev = _rows_of("xq", xq), xq.device
    E, N, K, pw, pws, po = _i8_weights(wq, ws, offsets, dev)
    pq = _addr("xq", xq, (torch.int8,), (T, K), dev)
    ps = _addr("xs", xs, (torch.float32,), (T,), dev)
    R, pt = _row_token(row_token, T, dev)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    given = out
    out, clear = _new_or_checked(out, (R, N), out_dtype or torch.bfloat16, tuple(_DT), xq)
    py = _addr("out", out, tuple(_DT), (R, N), dev)
    c = MoeMmCfg(R, N, K, E, T, 0, _DT[out.dtype], clear)
    _call("moe_mm_i8", dev.index, C.byref(c), pq, ps, pw, pws, po, pt, py)
    if given is not None:
        _written(given)
    return out


def _linear_bytes(c: MoeMmCfg, gathered: int) -> int:
    n = C.c_size_t(0)
    _check("moe_linear_i8_workspace_size", (_lib or load()).moe_linear_i8_workspace_size(C.byref(c), gathered, C.byref(n)))
    return n.value


def moe_linear_i8_workspace_size(rows: int, K: int, out_rows: Optional[int] = None) -> int:
    """Bytes of scratch moe_linear_i8 needs for x of `rows` rows, K inputs of w
    and, with row_token, `out_rows` rows of the result."""
    return _linear_bytes(MoeMmCfg(rows if out_rows is None else out_rows, 8, K, 1, rows, 0, 0, 0),
                         int(out_rows is not None))


def moe_linear_i8(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                  row_token: Optional[torch.Tensor] = None, swiglu: bool = False, out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None, work: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_mm_i8 of moe_quant_i8(x, swiglu): 16-bit activations (bfloat16 or
    float16) times int8 weights.  The result has x's type unless out_dtype or
    `out` says otherwise.  `work`: uint8 scratch of at least
    moe_linear_i8_workspace_size(...) bytes, allocated where absent and needed.
    Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_linear_i8", out, x, ws)
    (T, _), dev = _rows_of("x", x), x.device
    E, N, K, pw, pws, po = _i8_weights(wq, ws, offsets, dev)
    px = _addr("x", x, _16BIT, (T, 2 * K if swiglu else K), dev)
    R, pt = _row_token(row_token, T, dev)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    given = out
    out, clear = _new_or_checked(out, (R, N), out_dtype or x.dtype, tuple(_DT), x)
    py = _addr("out", out, tuple(_DT), (R, N), dev)
    c = MoeMmCfg(R, N, K, E, T, _DT[x.dtype], _DT[out.dtype], clear)
    if work is None:
        need = _linear_bytes(c, int(row_token is not None))
        work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    pk = None if work is None else _addr("work", work, (torch.uint8,), work.shape, dev)
    _call("moe_linear_i8", dev.index, C.byref(c), px, int(bool(swiglu)), pw, pws, po, pt, py, pk,
          0 if work is None else work.numel())
    if given is not None:
        _written(given)
    return out


def raw_call(name: str, *args) -> int:
    """Call a C entry point with raw ctypes arguments (for argument-check tests)."""
    return int(getattr(load(), name)(*args))
