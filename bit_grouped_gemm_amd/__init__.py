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
    moe_quant_mx4, moe_mm_mx4, moe_linear_mx4   (the same three in MXFP4: e2m1 codes, an e8m0 scale per 32)
    moe_layer_mm(x, topk_ids, topk_weights, w1, w2) -> out   (the whole layer for up to 64 tokens, 16-bit experts)
and in front of them
    moe_rms_norm(x, weight, residual=None) -> y, or (y, x + residual)   (differentiable)
    moe_rms_norm_quant(x, weight, residual=None, fmt=QFMT_E4M3) -> (codes, scales, y, sum)

The layer's GEMM entry points read expert weights in the tiled layout: convert the
canonical row-major tensors once with moe_prepack_weights(cfg, weights)
(a one-time step at weight load).
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import functools
import operator
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
QFMT_E4M3 = 0  # moe_rms_norm_quant's codes
QFMT_I8 = 1
QFMT_MXFP4 = 2
RATE_E2M1_E2M1 = 16  # moe_mfma_rate's e2m1 x e2m1 operand pair
RATE_E2M1_E2M1_32 = 17  # the same in the 32x32x64 form

EXPORTS = ("moe_workspace_size", "moe_permute", "moe_grouped_gemm1_swiglu", "moe_grouped_gemm2",
           "moe_combine", "moe_layer", "moe_layer_static", "moe_layer_persistent", "moe_layer_persistent_spin_limit",
           "moe_prepack_weights",
           "moe_stream_read",
           "moe_mfma_rate", "moe_encode_e4m3", "moe_route", "moe_route_workspace_size", "moe_status_str",
           "moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad",
           "moe_grouped_mm_wgrad_workspace_size", "moe_quant_i8", "moe_mm_i8",
           "moe_linear_i8", "moe_linear_i8_workspace_size",
           "moe_quant_mx4", "moe_mm_mx4", "moe_linear_mx4", "moe_linear_mx4_workspace_size",
           "moe_layer_mm", "moe_layer_mm_workspace_size",
           "moe_rms_norm", "moe_rms_norm_quant", "moe_rms_norm_backward", "moe_rms_norm_backward_workspace_size")

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


class MoeFewCfg(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("T", "H", "I", "E", "topk", "dtype")]


class MoeNormCfg(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("R", "K", "dtype", "weight_dtype", "fmt", "group")] + [("eps", C.c_float)]


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
    L.moe_quant_mx4.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int, vp, vp, vp, vp]
    L.moe_mm_mx4.argtypes = [mmp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_linear_mx4_workspace_size.argtypes = [mmp, C.c_int, C.POINTER(sz)]
    L.moe_linear_mx4.argtypes = [mmp, vp, C.c_int, vp, vp, vp, vp, vp, vp, sz, vp]
    fewp = C.POINTER(MoeFewCfg)
    L.moe_layer_mm.argtypes = [fewp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_layer_mm_workspace_size.argtypes = [fewp, C.POINTER(sz)]
    normp = C.POINTER(MoeNormCfg)
    L.moe_rms_norm.argtypes = [normp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_rms_norm_quant.argtypes = [normp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_rms_norm_backward.argtypes = [normp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_rms_norm_backward_workspace_size.argtypes = [normp, C.POINTER(sz)]
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
        if forward_ad._current_level >= 0:
            _refuse_tangents("moe_grouped_mm's gradient", dy)
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


def _beside(name, given, like):
    """An output of a checked operand's own kind and its address: a new one, or the caller's."""
    if given is None:
        out = torch.empty_like(like)
        return out, out.data_ptr() or None
    return given, _addr(name, given, (like.dtype,), like.shape, like.device)


# The calls' structs, by their values: put together once per shape.  The values are Python's own numbers
# (a tensor would be kept as itself, with the number it had at first).
_int = operator.index


def _struct(kind, values):
    c = kind(*values)
    for (name, ctype), v in zip(kind._fields_, values):
        if ctype is C.c_int32 and getattr(c, name) != v:
            raise ValueError(f"{name}: {v} does not fit 32 bits")
    return C.byref(c)


@functools.lru_cache(maxsize=1024)
def _mm_cfg(*values):
    return _struct(MoeMmCfg, values)


@functools.lru_cache(maxsize=1024)
def _few_cfg(*values):
    return _struct(MoeFewCfg, values)


@functools.lru_cache(maxsize=1024)
def _norm_cfg(*values):
    return _struct(MoeNormCfg, values)


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(name: str, cfg, *more) -> int:
    """The workspace size that entry point `name` gives for a cached struct."""
    n = C.c_size_t(0)
    _check(name, getattr(_lib or load(), name)(cfg, *more, C.byref(n)))
    return n.value


# ------------------------------------------------------------------ row-major MXFP4
def moe_quant_mx4(x: torch.Tensor, swiglu: bool = False, codes: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """MXFP4 codes uint8 [R, K / 2] (two e2m1 per byte, the even column in the low
    half) and e8m0 scales uint8 [R, K / 32] of the rows of x [R, K] (bfloat16 or
    float16; activations or weights), or of silu(gate) * up with x [R, 2 K] =
    gate | up where `swiglu`.  A block with an infinity or NaN gets the scale 255,
    e8m0's NaN.  Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_quant_mx4", None, x)
    (R, width), dev = _rows_of("x", x), x.device
    if swiglu and width % 2:
        raise ValueError(f"x: {width} columns do not split into gate and up")
    K = width // 2 if swiglu else width
    px = _addr("x", x, _16BIT, (R, width), dev)
    given = codes, scales
    if codes is None:
        codes = torch.empty(R, K // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(R, K // 32, dtype=torch.uint8, device=dev)
    pq = _addr("codes", codes, (torch.uint8,), (R, K // 2), dev)
    ps = _addr("scales", scales, (torch.uint8,), (R, K // 32), dev)
    _call("moe_quant_mx4", dev.index, R, K, _DT[x.dtype], int(bool(swiglu)), px, pq, ps)
    for t in given:
        if t is not None:
            _written(t)
    return codes, scales


def _mx4_weights(wq, ws, offsets, dev):
    """E, N, K and the addresses of MXFP4 weights [E, N, K / 2], or [N, K / 2] (dense:
    no offsets), of their scales and of the offsets."""
    if wq.dim() != (2 if offsets is None else 3):
        raise ValueError(f"wq: [N, K / 2] without offsets, [E, N, K / 2] with offsets; got {tuple(wq.shape)}")
    E, N, half = (1, *wq.shape) if offsets is None else wq.shape
    if max(wq.shape) > 0x3FFFFFFF:
        raise ValueError(f"wq: shape {tuple(wq.shape)}, sizes are at most 2^30 - 1")
    pw = _addr("wq", wq, (torch.uint8,), wq.shape, dev)
    ps = _addr("ws", ws, (torch.uint8,), (*wq.shape[:-1], half // 16), dev)
    po = None if offsets is None else _addr("offsets", offsets, (torch.int32,), (E + 1,), dev)
    return E, N, 2 * half, pw, ps, po


def moe_mm_mx4(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, row_token: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y[r] = x[t] @ w[e]^T with both operands in MXFP4 (moe_quant_mx4's codes and
    scales), fp32 sums.

    Dense: wq [N, K / 2], ws [N, K / 32], every row of xq.  Grouped: wq [E, N, K / 2],
    ws [E, N, K / 32] and offsets int32 [E + 1]; with row_token int32 [R]
    (moe_permute's) row r of the result takes row t = row_token[r] of xq, else t = r.
    The result [R, N] is bfloat16 (default), float16 or float32; rows of no
    group are zeros in a new result and stay as they are in a caller's `out`.
    Not differentiable: outputs that need a gradient are refused."""
    _refuse_derivatives("moe_mm_mx4", out)
    (T, width), dev = _rows_of("xq", xq), xq.device
    E, N, K, pw, pws, po = _mx4_weights(wq, ws, offsets, dev)
    pq = _addr("xq", xq, (torch.uint8,), (T, K // 2), dev)
    ps = _addr("xs", xs, (torch.uint8,), (T, K // 32), dev)
    R, pt = _row_token(row_token, T, dev)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    given = out
    out, clear = _new_or_checked(out, (R, N), out_dtype or torch.bfloat16, tuple(_DT), xq)
    py = _addr("out", out, tuple(_DT), (R, N), dev)
    c = _mm_cfg(R, N, K, E, T, 0, _DT[out.dtype], clear)
    _call("moe_mm_mx4", dev.index, c, pq, ps, pw, pws, po, pt, py)
    if given is not None:
        _written(given)
    return out


def moe_linear_mx4_workspace_size(rows: int, K: int, out_rows: Optional[int] = None) -> int:
    """Bytes of scratch moe_linear_mx4 needs for x of `rows` rows, K inputs of w
    and, with row_token, `out_rows` rows of the result."""
    rows, K, out_rows = _int(rows), _int(K), None if out_rows is None else _int(out_rows)
    return _scratch_bytes("moe_linear_mx4_workspace_size",
                          _mm_cfg(rows if out_rows is None else out_rows, 8, K, 1, rows, 0, 0, 0),
                          int(out_rows is not None))


def moe_linear_mx4(x: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                   row_token: Optional[torch.Tensor] = None, swiglu: bool = False, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, work: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_mm_mx4 of moe_quant_mx4(x, swiglu): 16-bit activations (bfloat16 or
    float16) times MXFP4 weights.  The result has x's type unless out_dtype or
    `out` says otherwise.  `work`: uint8 scratch of at least
    moe_linear_mx4_workspace_size(...) bytes, allocated where absent and needed.
    Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_linear_mx4", out, x)
    (T, _), dev = _rows_of("x", x), x.device
    E, N, K, pw, pws, po = _mx4_weights(wq, ws, offsets, dev)
    px = _addr("x", x, _16BIT, (T, 2 * K if swiglu else K), dev)
    R, pt = _row_token(row_token, T, dev)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    given = out
    out, clear = _new_or_checked(out, (R, N), out_dtype or x.dtype, tuple(_DT), x)
    py = _addr("out", out, tuple(_DT), (R, N), dev)
    c = _mm_cfg(R, N, K, E, T, _DT[x.dtype], _DT[out.dtype], clear)
    if work is None:
        need = _scratch_bytes("moe_linear_mx4_workspace_size", c, int(row_token is not None))
        work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    pk = None if work is None else _addr("work", work, (torch.uint8,), work.shape, dev)
    _call("moe_linear_mx4", dev.index, c, px, int(bool(swiglu)), pw, pws, po, pt, py, pk,
          0 if work is None else work.numel())
    if given is not None:
        _written(given)
    return out


# ------------------------------------------------------------------ the layer for a few tokens
def moe_layer_mm_workspace_size(T: int, H: int, I: int, E: int, topk: int) -> int:
    """Bytes of scratch moe_layer_mm needs for T tokens."""
    return _scratch_bytes("moe_layer_mm_workspace_size", _few_cfg(*map(_int, (T, H, I, E, topk)), 0))


def moe_layer_mm(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, w1: torch.Tensor,
                 w2: torch.Tensor, out: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, H] = sum over j of topk_weights[t, j] * w2[e] (silu(g) * u) with (g, u) =
    w1[e] x[t] and e = topk_ids[t, j], for up to 64 tokens: the whole expert layer on
    16-bit row-major weights in two launches (three where that pays).

    x [T, H], w1 [E, 2 I, H] (gate rows first) and w2 [E, H, I] are all bfloat16 or all
    float16; topk_ids int32 and topk_weights float32 [T, topk] as moe_route gives
    them.  Ids outside [0, E) are masked slots.  h = silu(g) * u has 17 bits in
    bfloat16 and 21 in float16, down to 2^-24 there; past float16's 65504 it is
    infinite, and with it the token's result.  `ws`: uint8 scratch of at least
    moe_layer_mm_workspace_size(...) bytes, allocated where absent; calls that share
    one must not overlap.  An always-on shared expert is one more matrix pair behind
    the others, named by one more slot of weight 1 (from 33 tokens on its weights
    are read twice).  For more tokens use moe_grouped_mm
    (MOE_ERR_UNSUPPORTED here).  Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_layer_mm", out, x, topk_weights)
    _refuse_derivatives("moe_layer_mm", None, w1, w2)
    (T, H), dt, dev = _rows_of("x", x), x.dtype, x.device
    topk = _rows_of("topk_ids", topk_ids)[1]
    E, two, _ = _matrices(w1)
    if two % 2:
        raise ValueError(f"w1: {two} rows do not split into gate and up")
    I = two // 2
    px = _addr("x", x, _16BIT, (T, H), dev)
    pi = _addr("topk_ids", topk_ids, (torch.int32,), (T, topk), dev)
    pt = _addr("topk_weights", topk_weights, (torch.float32,), (T, topk), dev)
    p1 = _addr("w1", w1, (dt,), (E, two, H), dev)
    p2 = _addr("w2", w2, (dt,), (E, H, I), dev)
    given = out
    out, po = _beside("out", out, x)
    c = _few_cfg(T, H, I, E, topk, _DT[dt])
    if ws is None:
        nb = _scratch_bytes("moe_layer_mm_workspace_size", c)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        pk = ws.data_ptr() or None
    else:
        pk, nb = _addr("ws", ws, (torch.uint8,), ws.shape, dev), ws.numel()
    _call("moe_layer_mm", dev.index, c, px, pi, pt, p1, p2, po, pk, nb)
    if given is not None:
        _written(given)
    return out


# ------------------------------------------------------------------ RMS norm
def _norm_operands(x, weight, residual, eps, fmt=0, group=0):
    """The call's cfg, sizes and the addresses of x, residual and weight."""
    (R, K), dt, dev = _rows_of("x", x), x.dtype, x.device
    px = _addr("x", x, _16BIT, (R, K), dev)
    pr = None if residual is None else _addr("residual", residual, (dt,), (R, K), dev)
    pw = _addr("weight", weight, (dt, torch.float32), (K,), dev)
    return _norm_cfg(R, K, _DT[dt], _DT[weight.dtype], fmt, group, eps), R, K, px, pr, pw


def _rms_norm(x, weight, residual, eps, out=None, sum_out=None, want_rstd=False):
    if residual is None and sum_out is not None:
        raise ValueError("sum_out needs a residual")
    c, R, K, px, pr, pw = _norm_operands(x, weight, residual, eps)
    y, py = _beside("out", out, x)
    s = ps = rstd = None
    if residual is not None:
        s, ps = _beside("sum_out", sum_out, x)
        if R and py == ps:
            raise ValueError("out and sum_out are the same tensor")
    if want_rstd:
        rstd = torch.empty(R, dtype=torch.float32, device=x.device)
    _call("moe_rms_norm", x.device.index, c, px, pr, pw, py, ps,
          None if rstd is None else rstd.data_ptr() or None)
    for t in (out, sum_out if residual is not None else None):
        if t is not None:
            _written(t)
    return y, s, rstd


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, s, rstd = _rms_norm(x, weight, residual, eps, want_rstd=True)
        ctx.eps, ctx.saw = eps, (x.shape, x.dtype, weight.dtype, x.device)
        ctx.save_for_backward(x if residual is None else s, weight, rstd)
        return y if residual is None else (y, s)

    @staticmethod
    def backward(ctx, dy, ds=None):
        # (the wrapper only matters where a graph of the gradients is asked for, and takes as long as a launch)
        return (_rms_norm_grads_once if _grad_enabled() else _rms_norm_grads)(ctx, dy, ds)


def _rms_norm_grads(ctx, dy, ds):
    s, weight, rstd = ctx.saved_tensors
    need_x, need_w, need_r, _ = ctx.needs_input_grad
    if dy is None:  # only the sum was used: its gradient is x's and the residual's
        return ds if need_x else None, None, ds if need_r else None, None
    if forward_ad._current_level >= 0:
        _refuse_tangents("moe_rms_norm's gradient", dy, ds)
    shape, dt, wdt, dev = ctx.saw
    R, K = shape
    dy, pd = _back("dy", dy, dt, shape, dev)
    pg = None
    if ds is not None:
        ds, pg = _back("the sum's gradient", ds, dt, shape, dev)
    s, ps = _back("sum", s, dt, shape, dev)
    weight, pw = _back("weight", weight, wdt, (K,), dev)
    rstd, pr = _back("rstd", rstd, torch.float32, (R,), dev)
    c = _norm_cfg(R, K, _DT[dt], _DT[wdt], 0, 0, ctx.eps)
    dx = dw = work = None
    need = 0
    if need_x or need_r:
        dx = torch.empty(shape, dtype=dt, device=dev)
    if need_w:
        dw = torch.empty(K, dtype=wdt, device=dev)
        need = _scratch_bytes("moe_rms_norm_backward_workspace_size", c)
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=dev)
    _call("moe_rms_norm_backward", dev.index, c, pd, pg, ps, pr, pw,
          None if dx is None else dx.data_ptr() or None, None if dw is None else dw.data_ptr() or None,
          None if work is None else work.data_ptr(), need)
    return dx if need_x else None, dw, dx if need_r else None, None


_rms_norm_grads_once = torch.autograd.function.once_differentiable(_rms_norm_grads)


def _back(name, t, dtype, shape, dev):
    """A tensor that autograd hands to a backward pass, as the kernels take it, and its address.  It need not be
    the one that forward saw: a hook may have made another of it, or its data may have been
    replaced, and a gradient may be an expanded or an unaligned view."""
    if t.dtype != dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"moe_rms_norm's gradient: {name} is {t.dtype} {tuple(t.shape)} on {t.device} now, "
                         f"was {dtype} {tuple(shape)} on {dev}")
    p = t.data_ptr()
    if p % 16 or not t.is_contiguous():
        t = t.clone(memory_format=torch.contiguous_format)
        p = t.data_ptr()
    return t, p or None


def _rms_norm_backward(dy, dsum, s, rstd, weight, eps, dx, dw, work):
    (R, K), dt, dev = _rows_of("dy", dy), dy.dtype, dy.device
    pd = _addr("dy", dy, _16BIT, (R, K), dev)
    pg = None if dsum is None else _addr("dsum", dsum, (dt,), (R, K), dev)
    ps = _addr("sum", s, (dt,), (R, K), dev)
    pr = _addr("rstd", rstd, (torch.float32,), (R,), dev)
    pw = _addr("weight", weight, (dt, torch.float32), (K,), dev)
    px = None if dx is None else _addr("dx", dx, (dt,), (R, K), dev)
    pdw = None if dw is None else _addr("dweight", dw, (weight.dtype,), (K,), dev)
    c = _norm_cfg(R, K, _DT[dt], _DT[weight.dtype], 0, 0, eps)
    if work is None and dw is not None:
        need = _scratch_bytes("moe_rms_norm_backward_workspace_size", c)
        work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    pk = None if work is None else _addr("work", work, (torch.uint8,), work.shape, dev)
    _call("moe_rms_norm_backward", dev.index, c, pd, pg, ps, pr, pw, px, pdw, pk,
          0 if work is None else work.numel())


def moe_rms_norm_backward_workspace_size(R: int, K: int) -> int:
    """Bytes of scratch moe_rms_norm_backward needs for the gradient of the weight."""
    return _scratch_bytes("moe_rms_norm_backward_workspace_size", _norm_cfg(_int(R), _int(K), 0, 0, 0, 0, 1.0))


def moe_rms_norm_backward(dy: torch.Tensor, dsum: Optional[torch.Tensor], sum: torch.Tensor, rstd: torch.Tensor,
                          weight: torch.Tensor, eps: float = 1e-6,
                          work: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of moe_rms_norm: `sum` [R, K] is what was normalised, `rstd`
    float32 [R] is 1 / sqrt(mean(sum^2) + eps), `dsum` (or None) the gradient that
    reaches the sum by itself.  dx is the residual's gradient too.  `work`: uint8
    scratch of at least moe_rms_norm_backward_workspace_size(R, K) bytes,
    allocated where absent.  Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_rms_norm_backward", dsum, dy, sum)
    _refuse_derivatives("moe_rms_norm_backward", None, rstd, weight)
    dx, dw = torch.empty_like(sum), torch.empty_like(weight)
    _rms_norm_backward(dy, dsum, sum, rstd, weight, float(eps), dx, dw, work)
    return dx, dw


def moe_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None):
    """y [R, K] = s / sqrt(mean(s^2) + eps) * weight for the rows of s = x +
    residual; returns y, or (y, s) where there is a residual.

    x and residual [R, K] are bfloat16 or float16 (K a multiple of 8 up to
    16384), weight [K] is of their type or float32, eps 1e-30 to 1.  s is rounded to their type
    before it is normalised: it is what the residual stream carries on.  `out` and
    `sum_out` receive y and s; `sum_out` may be x or residual itself.  All tensors
    are contiguous and on one GPU.

    Differentiable with respect to x, weight and residual (once; not with `out`
    or `sum_out`).  Operands with a forward-mode tangent are refused.  In a
    graph, capture forward and backward together, while no earlier result computed
    from the same leaves is kept."""
    eps = float(eps)
    if forward_ad._current_level >= 0:
        _refuse_tangents("moe_rms_norm", x, weight, residual, out, sum_out)
    if _grad_enabled():
        if x.requires_grad or weight.requires_grad or residual is not None and residual.requires_grad:
            if out is not None or sum_out is not None:
                raise ValueError("moe_rms_norm: out and sum_out cannot be given where a gradient is needed")
            return _RmsNorm.apply(x, weight, residual, eps)
        _refuse_derivatives("moe_rms_norm with out", out, sum_out)
    y, s, _ = _rms_norm(x, weight, residual, eps, out, sum_out)
    return y if residual is None else (y, s)


def moe_rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                       eps: float = 1e-6, fmt: int = QFMT_E4M3, group: int = 128, want_y: bool = False,
                       sum_out: Optional[torch.Tensor] = None):
    """moe_rms_norm with quantised rows: (codes, scales, y, sum).

    fmt QFMT_E4M3: codes uint8 [R, K] and float32 scales [R, K / group], group 32
    or 128 (moe_grouped_gemm1_swiglu takes them for xq and xs; moe_permute, which
    gives it the rest, quantises all the same); QFMT_I8:
    int8 [R, K] and float32 [R] (moe_mm_i8's); QFMT_MXFP4: uint8 [R, K / 2] and
    [R, K / 32] (moe_mm_mx4's).  y is the 16-bit result, for the router, or None
    without `want_y`; sum is x + residual, or None without a residual.  `sum_out` may
    be x or residual itself.  Not differentiable: operands that need a gradient are refused."""
    _refuse_derivatives("moe_rms_norm_quant", residual, x, weight)
    _refuse_derivatives("moe_rms_norm_quant", sum_out)
    if residual is None and sum_out is not None:
        raise ValueError("sum_out needs a residual")
    fmt, group = _int(fmt), _int(group)
    c, R, K, px, pr, pw = _norm_operands(x, weight, residual, float(eps), fmt, group)
    dev = x.device
    y = py = s = ps = None
    if want_y:
        y, py = _beside("y", None, x)
    if residual is not None:
        s, ps = _beside("sum_out", sum_out, x)
    if fmt == QFMT_MXFP4:
        codes = torch.empty(R, K // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(R, K // 32, dtype=torch.uint8, device=dev)
    elif fmt == QFMT_I8:
        codes = torch.empty(R, K, dtype=torch.int8, device=dev)
        scales = torch.empty(R, dtype=torch.float32, device=dev)
    else:
        codes = torch.empty(R, K, dtype=torch.uint8, device=dev)
        scales = torch.empty(R, K // max(group, 1), dtype=torch.float32, device=dev)
    _call("moe_rms_norm_quant", dev.index, c, px, pr, pw, py, ps, codes.data_ptr() or None,
          scales.data_ptr() or None)
    if s is not None and sum_out is not None:
        _written(sum_out)
    return codes, scales, y, s


def raw_call(name: str, *args) -> int:
    """Call a C entry point with raw ctypes arguments (for argument-check tests)."""
    return int(getattr(load(), name)(*args))
