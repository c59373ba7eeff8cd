"""Thin Python binding of libmoe_mi355x.so (the C ABI in include/moe_mi355x.h).

Argument marshalling only: every step of the layer runs in the library's HIP kernels.  torch is
used for device memory (output and workspace tensors) and for the current HIP stream.  If the
library is not built this module raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_MI355X_LIB may point at another build of the same library (e.g. to compare two builds).
LIB_PATH = os.environ.get("MOE_MI355X_LIB", os.path.join(_PKG, "libmoe_mi355x.so"))

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
DTYPE_BF16, DTYPE_FP8, DTYPE_MXFP4, DTYPE_MXFP4_A8, DTYPE_INT8 = 0, 1, 2, 3, 4
CONFIG_AUTO, CONFIG_STREAM, CONFIG_MFMA, CONFIG_FUSED = -1, 0, 1, 2
FUSED_SYNC_BYTES = 36864    # the fused single-token launch's counters at the workspace's start
CONFIG_POLICY0, NUM_POLICIES = 16, 8  # config = 16 + i forces selection policy i (bf16)
LAYOUT_ROW_MAJOR, LAYOUT_TILED = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
SCALE_BF16, SCALE_FP16 = 0, 1

_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("has_shared", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("config", ctypes.c_int32)]


WEIGHT_POINTERS = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
                   "sh_gate", "sh_up", "sh_down", "s_sh_gate", "s_sh_up", "s_sh_down",
                   "e_gate", "e_up", "e_down")


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_POINTERS] + [("layout", ctypes.c_int32)]


class Scoring(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "groups", "top_groups", "group_top", "renorm")] + [
        ("scale", ctypes.c_float)]


class Block(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("post_weight", "gate", "pre_weight")] + [
        ("gate_per_token", ctypes.c_int32)] + [
        (n, ctypes.c_float) for n in ("residual_scale", "branch_scale", "eps")]


class W4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scales", "zeros")] + [
        (n, ctypes.c_int32) for n in ("N", "K", "group", "scale_dtype", "layout")]


class Routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_ids", "topk_w", "counts", "offsets", "perm_src", "slot_dst", "eeff", "policy")]


class MoEError(RuntimeError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    """Loads the library (after torch, so both share torch's HIP runtime)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoEError(f"{LIB_PATH} is not built; run `python -m mixture_experts_layer_top_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_route": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp]),
            "moe_permute": (_i, [_vp, _i, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _sz, _vp]),
            "moe_permute_workspace_bytes": (_sz, [_i, _i, _i]),
            "moe_quant_act": (_i, [_vp, _i, _i, _vp, _vp, _vp]),
            "moe_quant_act_mx": (_i, [_vp, _i, _i, _vp, _vp, _vp]),
            "moe_grouped_ffn": (_i, [ctypes.POINTER(Problem), _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(Weights), _vp, _vp, _sz, _vp]),
            "moe_grouped_ffn_workspace_bytes": (_sz, [ctypes.POINTER(Problem)]),
            "moe_combine": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
            "moe_layer": (_i, [ctypes.POINTER(Problem), _vp, _vp, ctypes.POINTER(Weights), _vp,
                               ctypes.POINTER(Routing), _vp, _sz, _vp]),
            "moe_layer_workspace_bytes": (_sz, [ctypes.POINTER(Problem)]),
            "moe_layer_traced": (_i, [ctypes.POINTER(Problem), _vp, _vp, ctypes.POINTER(Weights), _vp,
                                      ctypes.POINTER(Routing), _vp, _sz, ctypes.POINTER(_vp), _i, _vp]),
            "moe_status_string": (ctypes.c_char_p, [_i]),
            "moe_mxfp4_tile": (_i, [_vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp]),
            "moe_fp8_tile": (_i, [_vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp]),
            "moe_layer_noalloc": (_i, [ctypes.POINTER(Problem), _vp, _vp, ctypes.POINTER(Weights),
                                       _vp, ctypes.POINTER(Routing), _vp]),
            "moe_quant_act_i8": (_i, [_vp, _i, _i, _vp, _vp, _vp]),
            "moe_gemm_i8": (_i, [_vp, _vp, _i, _vp, _vp, _i, _i, _vp, _vp]),
            "moe_rmsnorm": (_i, [_vp, _vp, _vp, _f, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
            "moe_rmsnorm_grad": (_i, [_vp, _vp, _vp, _vp, _f, _i, _i, _vp, _vp, _vp, _sz, _vp]),
            "moe_rmsnorm_grad_workspace_bytes": (_sz, [_i, _i]),
            "moe_route_grad": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
            "moe_combine_grad": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
            "moe_permute_grad": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
            "moe_route_scored": (_i, [_vp, _vp, _i, _i, _i, ctypes.POINTER(Scoring), _vp, _vp, _vp]),
            "moe_route_scored_grad": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, ctypes.POINTER(Scoring), _vp, _vp]),
            "moe_block_norm": (_i, [ctypes.POINTER(Block), _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
            "moe_block_norm_grad": (_i, [ctypes.POINTER(Block), _vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _sz, _vp]),
            "moe_block_norm_grad_workspace_bytes": (_sz, [_i, _i]),
            "moe_w4_tile": (_i, [ctypes.POINTER(W4), _vp, _vp, _vp, _vp]),
            "moe_gemm_w4": (_i, [_vp, _i, ctypes.POINTER(W4), ctypes.POINTER(W4), _vp, _vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


EXPORTED = ("moe_route", "moe_permute", "moe_permute_workspace_bytes", "moe_quant_act",
            "moe_quant_act_mx",
            "moe_grouped_ffn", "moe_grouped_ffn_workspace_bytes", "moe_combine", "moe_layer",
            "moe_layer_workspace_bytes", "moe_layer_traced", "moe_status_string", "moe_mxfp4_tile",
            "moe_fp8_tile", "moe_layer_noalloc", "moe_quant_act_i8", "moe_gemm_i8", "moe_rmsnorm",
            "moe_rmsnorm_grad", "moe_rmsnorm_grad_workspace_bytes", "moe_route_grad",
            "moe_combine_grad", "moe_permute_grad", "moe_route_scored", "moe_route_scored_grad",
            "moe_block_norm", "moe_block_norm_grad", "moe_block_norm_grad_workspace_bytes", "moe_w4_tile",
            "moe_gemm_w4")

NOALLOC_SCRATCH_BYTES = 128 << 20  # MOE_NOALLOC_SCRATCH_BYTES

TRACE_EVENTS = 8
TRACE_PHASES = ("route", "permute", "quant", "select", "gate_up", "down", "combine")


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        raise MoEError(f"{what}: {lib().moe_status_string(status).decode()}")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _dev(t):
    if not t.is_cuda:
        raise MoEError("tensors must live on the GPU")
    return t.device


@dataclass
class ExpertWeights:
    """Device tensors of the expert weights in the library's storage layout."""
    gate: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor
    s_gate: torch.Tensor | None = None
    s_up: torch.Tensor | None = None
    s_down: torch.Tensor | None = None
    sh_gate: torch.Tensor | None = None
    sh_up: torch.Tensor | None = None
    sh_down: torch.Tensor | None = None
    s_sh_gate: torch.Tensor | None = None
    s_sh_up: torch.Tensor | None = None
    s_sh_down: torch.Tensor | None = None
    e_gate: torch.Tensor | None = None  # mxfp4: uint8 E8M0 scales [E, f, d/32] / [E, d, f/32]
    e_up: torch.Tensor | None = None
    e_down: torch.Tensor | None = None
    act_mx8: bool = False  # mxfp4 weights: quantise activations (and h) to MXFP8 (MOE_DTYPE_MXFP4_A8)

    def struct(self) -> Weights:
        w = Weights()
        for name in WEIGHT_POINTERS:
            key = {"w_gate": "gate", "w_up": "up", "w_down": "down"}.get(name, name)
            setattr(w, name, _ptr(getattr(self, key)))
        w.layout = LAYOUT_ROW_MAJOR
        if self.wdtype != DTYPE_BF16:
            # fp8 / int8 / mxfp4 bytes count as tiled only if every weight tensor came from fp8_tile,
            # int8_tile or mxfp4_tile (the library rejects row-major bytes of these formats)
            mats = [self.gate, self.up, self.down] + (
                [self.sh_gate, self.sh_up, self.sh_down] if self.has_shared else [])
            if all(getattr(t, "_moe_tiled", False) for t in mats):
                w.layout = LAYOUT_TILED
        return w

    @property
    def wdtype(self) -> int:
        if self.e_gate is not None:
            return DTYPE_MXFP4_A8 if self.act_mx8 else DTYPE_MXFP4
        if self.gate.dtype == torch.int8:
            return DTYPE_INT8
        return DTYPE_FP8 if self.gate.dtype == torch.uint8 else DTYPE_BF16

    @property
    def fp8(self) -> bool:
        return self.wdtype == DTYPE_FP8

    @property
    def d_model(self) -> int:
        """d from the gate weights' last dim (two mxfp4 elements per byte)."""
        return self.gate.shape[2] * (2 if self.wdtype in (DTYPE_MXFP4, DTYPE_MXFP4_A8) else 1)

    @property
    def has_shared(self) -> bool:
        return self.sh_gate is not None


def problem(T, d, f, E, k, fp8=False, shared_f=0, config=CONFIG_AUTO, wdtype=None) -> Problem:
    if wdtype is None:
        wdtype = DTYPE_FP8 if fp8 else DTYPE_BF16
    return Problem(T, d, f, E, k, wdtype, 1 if shared_f else 0, shared_f, config)


# ------------------------------------------------------------------------------------------------
# entry points
# ------------------------------------------------------------------------------------------------

def route(logits: torch.Tensor, k: int):
    T, E = logits.shape
    dev = _dev(logits)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _check(lib().moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream()), "moe_route")
    return ids, w


def permute(ids: torch.Tensor, E: int, x: torch.Tensor | None = None,
            x_scale: torch.Tensor | None = None):
    """Returns counts, offsets, perm_src, slot_dst (and x_perm, x_perm_scale if x is given).
    x: bf16 [T, d] as int16 bits, e4m3 [T, d] uint8 (with x_scale [T, d/128]) or int8 [T, d] (with
    x_scale [T])."""
    T, k = ids.shape
    dev = _dev(ids)
    n = T * k
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm_src = torch.empty(n, dtype=torch.int32, device=dev)
    slot_dst = torch.empty(n, dtype=torch.int32, device=dev)
    ws = torch.empty(max(1, lib().moe_permute_workspace_bytes(T, E, k)), dtype=torch.uint8, device=dev)
    xp = xps = None
    d = 0
    act = DTYPE_BF16
    if x is not None:
        d = x.shape[1]
        act = {torch.uint8: DTYPE_FP8, torch.int8: DTYPE_INT8}.get(x.dtype, DTYPE_BF16)
        xp = torch.empty((n, d), dtype=x.dtype, device=dev)
        if x_scale is not None:
            shape = (n,) if act == DTYPE_INT8 else (n, d // 128)
            xps = torch.empty(shape, dtype=torch.float32, device=dev)
    _check(lib().moe_permute(_ptr(ids), T, E, k, _ptr(x), _ptr(x_scale), d, act, _ptr(counts),
                             _ptr(offsets), _ptr(perm_src), _ptr(slot_dst), _ptr(xp), _ptr(xps),
                             _ptr(ws), ws.numel(), _stream()), "moe_permute")
    return counts, offsets, perm_src, slot_dst, xp, xps


def mxfp4_tile(w: torch.Tensor) -> torch.Tensor:
    """Row-major MXFP4 bytes [..., rows, cols/2] (uint8) -> the library's tiled layout (same shape;
    every leading dimension folds into the rows)."""
    w = w.contiguous()
    out = torch.empty_like(w)
    rows = w.numel() // w.shape[-1]
    _check(lib().moe_mxfp4_tile(_ptr(w), _ptr(out), rows, 2 * w.shape[-1], _stream()),
           "moe_mxfp4_tile")
    out._moe_tiled = True
    return out


def fp8_tile(w: torch.Tensor) -> torch.Tensor:
    """Row-major fp8 weight bytes [..., rows, cols] (uint8) -> the library's tiled layout."""
    w = w.contiguous()
    out = torch.empty_like(w)
    rows = w.numel() // w.shape[-1]
    _check(lib().moe_fp8_tile(_ptr(w), _ptr(out), rows, w.shape[-1], _stream()), "moe_fp8_tile")
    out._moe_tiled = True
    return out


def quant_act(x: torch.Tensor):
    T, d = x.shape
    dev = _dev(x)
    xq = torch.empty((T, d), dtype=torch.uint8, device=dev)
    xs = torch.empty((T, d // 128), dtype=torch.float32, device=dev)
    _check(lib().moe_quant_act(_ptr(x), T, d, _ptr(xq), _ptr(xs), _stream()), "moe_quant_act")
    return xq, xs


def quant_act_mx(x: torch.Tensor):
    """bf16 [T, d] (int16 bits) -> MXFP8: e4m3 codes [T, d] and E8M0 scale codes [T, d/32]."""
    T, d = x.shape
    dev = _dev(x)
    xq = torch.empty((T, d), dtype=torch.uint8, device=dev)
    xe = torch.empty((T, d // 32), dtype=torch.uint8, device=dev)
    _check(lib().moe_quant_act_mx(_ptr(x), T, d, _ptr(xq), _ptr(xe), _stream()), "moe_quant_act_mx")
    return xq, xe


def grouped_ffn(x_perm, x_perm_scale, counts, offsets, weights: ExpertWeights, T: int, k: int,
                config: int = CONFIG_AUTO):
    n, d = x_perm.shape
    E = counts.shape[0]
    f = weights.gate.shape[1]
    p = problem(T, d, f, E, k, config=config, wdtype=weights.wdtype)
    dev = _dev(x_perm)
    y = torch.empty((n, d), dtype=torch.int16, device=dev)
    ws = torch.empty(max(1, lib().moe_grouped_ffn_workspace_bytes(ctypes.byref(p))),
                     dtype=torch.uint8, device=dev)
    w = weights.struct()
    _check(lib().moe_grouped_ffn(ctypes.byref(p), _ptr(x_perm), _ptr(x_perm_scale), _ptr(counts),
                                 _ptr(offsets), ctypes.byref(w), _ptr(y), _ptr(ws), ws.numel(),
                                 _stream()), "moe_grouped_ffn")
    return y


def combine(y_perm, slot_dst, topk_w, shared_y=None):
    T, k = topk_w.shape
    d = y_perm.shape[1]
    out = torch.empty((T, d), dtype=torch.int16, device=_dev(y_perm))
    _check(lib().moe_combine(_ptr(y_perm), _ptr(slot_dst), _ptr(topk_w), T, k, d, _ptr(shared_y),
                             _ptr(out), _stream()), "moe_combine")
    return out


# ------------------------------------------------------------------------------------------------
# int8 and 4-bit products, RMS norms, routing by scores, gradients
#
# bf16 tensors are torch.bfloat16 or their bits as torch.int16, like the rest of this module's; outputs
# take the input's choice.  Tensors must be contiguous and on one GPU, which need not be the current
# one: a call runs on that GPU's current stream.  (The layer's own steps above and Layer run on the
# current GPU, which has to be the tensors'.)  No call records anything for autograd: outputs never require
# grad, and a training step calls the gradients by name.  These calls are a few microseconds of GPU work at
# decode sizes, so what they do on the host counts: one pass of cheap checks per tensor, and the stream's
# handle without a Stream object (2 us).
# ------------------------------------------------------------------------------------------------

_BF16 = (torch.bfloat16, torch.int16)
_I8, _I32, _F32 = (torch.int8,), (torch.int32,), (torch.float32,)


def _arg(t, name, shape, dtypes, dev):
    """Checks a tensor: one of these types, this shape, contiguous, on GPU dev (-1: not checked here)."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return
    if t.dtype not in dtypes:
        raise MoEError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.shape != shape:
        raise MoEError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise MoEError(f"{name} must be contiguous")
    if dev >= 0:
        raise MoEError(f"{name} must live on GPU {dev}, not on {t.device}")


def _rows(t, name):
    if t.dim() != 2:
        raise MoEError(f"{name} must have two dimensions, not {t.dim()}")
    return t.shape


def _run(name, dev, *args):
    """One library call (tensors' addresses and numbers) on GPU dev's current stream."""
    if dev < 0:
        raise MoEError("tensors must live on the GPU")
    fn = getattr(lib(), name)
    if dev == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != MOE_OK:
        _check(st, name)


def quant_act_i8(x: torch.Tensor):
    """bf16 [T, d] -> int8 codes [T, d] and fp32 scales [T] (per token; or per channel of weights)."""
    T, d = _rows(x, "x")
    dev = x.get_device()
    _arg(x, "x", (T, d), _BF16, dev)
    xq = torch.empty_like(x, dtype=torch.int8)
    xs = x.new_empty(T, dtype=torch.float32)
    _run("moe_quant_act_i8", dev, x.data_ptr(), T, d, xq.data_ptr(), xs.data_ptr())
    return xq, xs


def int8_tile(w: torch.Tensor) -> torch.Tensor:
    """Row-major int8 weights [..., rows, cols] -> the library's tiled layout (moe_fp8_tile: the layout
    is the same for every one-byte format)."""
    if w.dtype != torch.int8:
        raise MoEError(f"w must be torch.int8, not {w.dtype}")
    _dev(w)
    with torch.cuda.device(w.get_device()):
        return fp8_tile(w)


def gemm_i8(xq: torch.Tensor, xs: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor):
    """bf16 [M, N] = (xq [M, K] * xs [M]) (w [N, K] * w_scale [N])^T; w from int8_tile."""
    (M, K), (N, _) = _rows(xq, "xq"), _rows(w, "w")
    dev = xq.get_device()
    _arg(xq, "xq", (M, K), _I8, dev)
    _arg(xs, "xs", (M,), _F32, dev)
    _arg(w, "w", (N, K), _I8, dev)
    _arg(w_scale, "w_scale", (N,), _F32, dev)
    if not getattr(w, "_moe_tiled", False):
        raise MoEError("w must come from int8_tile")
    y = xq.new_empty((M, N), dtype=torch.bfloat16)
    _run("moe_gemm_i8", dev, xq.data_ptr(), xs.data_ptr(), M, w.data_ptr(), w_scale.data_ptr(), N, K,
         y.data_ptr())
    return y


def _norm_outputs(x, T, d, act_dtype, want_y):
    """A norm call's (y, q, q_scale), None where not wanted, and their addresses."""
    y = q = qs = yp = qp = sp = None
    if want_y or act_dtype == DTYPE_BF16:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    if act_dtype != DTYPE_BF16:
        if act_dtype == DTYPE_INT8:
            q, qs = torch.empty_like(x, dtype=torch.int8), x.new_empty(T, dtype=torch.float32)
        elif act_dtype == DTYPE_FP8:
            q = torch.empty_like(x, dtype=torch.uint8)
            qs = x.new_empty((T, d // 128), dtype=torch.float32)
        else:
            q = torch.empty_like(x, dtype=torch.uint8)
            qs = x.new_empty((T, d // 32), dtype=torch.uint8)
        qp, sp = q.data_ptr(), qs.data_ptr()
    return y, q, qs, yp, qp, sp


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
            eps: float = 1e-6, act_dtype: int = DTYPE_BF16, want_y: bool = True):
    """RMS norm of h = x + residual.  Returns (h, y, q, q_scale): h is x itself without a residual, y is
    None when not wanted (8-bit outputs only), q and q_scale are y in the format act_dtype (DTYPE_FP8: e4m3
    uint8 and fp32 [T, d/128]; DTYPE_INT8: int8 and fp32 [T]: what permute and grouped_ffn take;
    DTYPE_MXFP4_A8: e4m3 and E8M0 uint8 [T, d/32], as quant_act_mx writes them, which no call here takes;
    DTYPE_BF16: None).  The outputs carry no autograd history (rmsnorm_grad is the gradient)."""
    T, d = _rows(x, "x")
    dev = x.get_device()
    _arg(x, "x", (T, d), _BF16, dev)
    _arg(weight, "weight", (d,), _BF16, dev)
    h, rp, hp = x, None, None
    if residual is not None:
        _arg(residual, "residual", (T, d), _BF16, dev)
        h = torch.empty_like(x)
        rp, hp = residual.data_ptr(), h.data_ptr()
    y, q, qs, yp, qp, sp = _norm_outputs(x, T, d, act_dtype, want_y)
    _run("moe_rmsnorm", dev, x.data_ptr(), rp, weight.data_ptr(), eps, T, d, act_dtype, hp, yp, qp, sp)
    return h, y, q, qs


def rmsnorm_grad(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                 dh: torch.Tensor | None = None, eps: float = 1e-6, want_dweight: bool = True):
    """Gradient of rmsnorm's y (and of h on the residual path, dh): (dx [T, d], dweight fp32 [d] or
    None).  dx is the gradient of x and of residual alike."""
    T, d = _rows(dy, "dy")
    dev = dy.get_device()
    _arg(dy, "dy", (T, d), _BF16, dev)
    _arg(h, "h", (T, d), _BF16, dev)
    _arg(weight, "weight", (d,), _BF16, dev)
    if dh is not None:
        _arg(dh, "dh", (T, d), _BF16, dev)
    dx = torch.empty_like(dy)
    dw = ws = None
    nws = 0
    if want_dweight:
        dw = dy.new_empty(d, dtype=torch.float32)
        nws = lib().moe_rmsnorm_grad_workspace_bytes(T, d)
        ws = dy.new_empty(nws, dtype=torch.uint8) if nws else None
    _run("moe_rmsnorm_grad", dev, dy.data_ptr(), _ptr(dh), h.data_ptr(), weight.data_ptr(), eps, T, d,
         dx.data_ptr(), _ptr(dw), _ptr(ws), nws)
    return dx, dw


def route_grad(ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor, E: int):
    """Gradient of route: ids, w, dw [T, k] -> dlogits fp32 [T, E]."""
    T, k = _rows(ids, "ids")
    dev = ids.get_device()
    _arg(ids, "ids", (T, k), _I32, dev)
    _arg(w, "w", (T, k), _F32, dev)
    _arg(dw, "dw", (T, k), _F32, dev)
    dl = w.new_empty((T, E))
    _run("moe_route_grad", dev, ids.data_ptr(), w.data_ptr(), dw.data_ptr(), T, E, k, dl.data_ptr())
    return dl


def combine_grad(dout: torch.Tensor, y_perm: torch.Tensor, slot_dst: torch.Tensor, topk_w: torch.Tensor):
    """Gradient of combine: (dy_perm [T*k, d], dtopk_w fp32 [T, k]); shared_y's is dout."""
    T, k = _rows(topk_w, "topk_w")
    d = _rows(dout, "dout")[1]
    dev = dout.get_device()
    _arg(dout, "dout", (T, d), _BF16, dev)
    _arg(topk_w, "topk_w", (T, k), _F32, dev)
    _arg(y_perm, "y_perm", (T * k, d), _BF16, dev)
    _arg(slot_dst, "slot_dst", (T * k,), _I32, dev)
    dy = torch.empty_like(y_perm)
    dw = torch.empty_like(topk_w)
    _run("moe_combine_grad", dev, dout.data_ptr(), y_perm.data_ptr(), slot_dst.data_ptr(),
         topk_w.data_ptr(), T, k, d, dy.data_ptr(), dw.data_ptr())
    return dy, dw


def permute_grad(dx_perm: torch.Tensor, slot_dst: torch.Tensor, k: int, add: torch.Tensor | None = None):
    """Gradient of permute's gather: dx [T, d] = each token's k rows of dx_perm summed (+ add)."""
    n, d = _rows(dx_perm, "dx_perm")
    if k < 1 or n % k:
        raise MoEError(f"dx_perm has {n} rows, not a multiple of k = {k}")
    T = n // k
    dev = dx_perm.get_device()
    _arg(dx_perm, "dx_perm", (n, d), _BF16, dev)
    _arg(slot_dst, "slot_dst", (n,), _I32, dev)
    if add is not None:
        _arg(add, "add", (T, d), _BF16, dev)
    dx = dx_perm.new_empty((T, d))
    _run("moe_permute_grad", dev, dx_perm.data_ptr(), slot_dst.data_ptr(), _ptr(add), T, k, d,
         dx.data_ptr())
    return dx


def _scoring(score, renorm, scale, groups=1, top_groups=1, group_top=1):
    return Scoring(score, groups, top_groups, group_top, 1 if renorm else 0, scale)


def route_scored(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: int = SCORE_SIGMOID,
                 groups: int = 1, top_groups: int = 1, group_top: int = 1, renorm: bool = True,
                 scale: float = 1.0):
    """Routing by scores (SCORE_SIGMOID, or SCORE_SOFTMAX over all experts): fp32 logits [T, E] and bias [E]
    -> ids int32 [T, k], the experts with the largest score + bias among the top_groups best of `groups`
    groups (valued by the sum of their group_top largest), and w fp32 [T, k], scale times their scores,
    renormalised over the k if wanted.  Experts with a logit of -inf are masked."""
    T, E = _rows(logits, "logits")
    dev = logits.get_device()
    _arg(logits, "logits", (T, E), _F32, dev)
    bp = None
    if bias is not None:
        _arg(bias, "bias", (E,), _F32, dev)
        bp = bias.data_ptr()
    ids = logits.new_empty((T, k), dtype=torch.int32)
    w = logits.new_empty((T, k))
    _run("moe_route_scored", dev, logits.data_ptr(), bp, T, E, k,
         _scoring(score, renorm, scale, groups, top_groups, group_top), ids.data_ptr(), w.data_ptr())
    return ids, w


def route_scored_grad(logits: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor,
                      score: int = SCORE_SIGMOID, renorm: bool = True, scale: float = 1.0):
    """Gradient of route_scored's weights: its logits [T, E], ids and w, and dw [T, k] -> dlogits fp32 [T, E]."""
    T, E = _rows(logits, "logits")
    k = _rows(ids, "ids")[1]
    dev = logits.get_device()
    _arg(logits, "logits", (T, E), _F32, dev)
    _arg(ids, "ids", (T, k), _I32, dev)
    _arg(w, "w", (T, k), _F32, dev)
    _arg(dw, "dw", (T, k), _F32, dev)
    dl = torch.empty_like(logits)
    _run("moe_route_scored_grad", dev, logits.data_ptr(), ids.data_ptr(), w.data_ptr(), dw.data_ptr(), T, E, k,
         _scoring(score, renorm, scale), dl.data_ptr())
    return dl


def _block(T, d, dev, pre_weight, post_weight, gate, residual_scale, branch_scale, eps):
    """The Block of a call and whether its gate has a row per token."""
    _arg(pre_weight, "pre_weight", (d,), _BF16, dev)
    if post_weight is not None:
        _arg(post_weight, "post_weight", (d,), _BF16, dev)
    rows = gate is not None and gate.dim() == 2
    if gate is not None:
        _arg(gate, "gate", (T, d) if rows else (d,), _BF16, dev)
    return Block(_ptr(post_weight), _ptr(gate), pre_weight.data_ptr(), 1 if rows else 0, residual_scale,
                 branch_scale, eps), rows


def block_norm(x: torch.Tensor, residual: torch.Tensor, pre_weight: torch.Tensor,
               post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               residual_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6,
               act_dtype: int = DTYPE_BF16, want_y: bool = True):
    """From a block's output x to the next block's input: h = residual_scale * residual + branch_scale * gate
    * (the RMS norm of x with post_weight, or x), y = the RMS norm of h with pre_weight.  gate: [d], or
    [T, d].  Returns (h, y, q, q_scale) as rmsnorm does."""
    T, d = _rows(x, "x")
    dev = x.get_device()
    _arg(x, "x", (T, d), _BF16, dev)
    _arg(residual, "residual", (T, d), _BF16, dev)
    b, _ = _block(T, d, dev, pre_weight, post_weight, gate, residual_scale, branch_scale, eps)
    h = torch.empty_like(x)
    y, q, qs, yp, qp, sp = _norm_outputs(x, T, d, act_dtype, want_y)
    _run("moe_block_norm", dev, b, x.data_ptr(), residual.data_ptr(), T, d, act_dtype, h.data_ptr(), yp, qp, sp)
    return h, y, q, qs


def block_norm_grad(dy: torch.Tensor, x: torch.Tensor, h: torch.Tensor, pre_weight: torch.Tensor,
                    dh: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
                    gate: torch.Tensor | None = None, residual_scale: float = 1.0, branch_scale: float = 1.0,
                    eps: float = 1e-6, want_sums: bool = True):
    """Gradient of block_norm's y (and of its h, dh), with the forward call's x and h.  Returns (dx,
    dresidual, dpre_weight, dpost_weight, dgate): [T, d] the first two, fp32 [d] the next two (None without a
    post_weight), dgate fp32 [d], [T, d] in the gate's type, or None without one.  Without want_sums those of
    [d] are None."""
    T, d = _rows(dy, "dy")
    dev = dy.get_device()
    for name, t in (("dy", dy), ("x", x), ("h", h)) + (() if dh is None else (("dh", dh),)):
        _arg(t, name, (T, d), _BF16, dev)
    b, rows = _block(T, d, dev, pre_weight, post_weight, gate, residual_scale, branch_scale, eps)
    dx, dres = torch.empty_like(dy), torch.empty_like(dy)
    dpre = dpost = dgate = ws = None
    nws = 0
    if rows:
        dgate = torch.empty_like(gate)
    if want_sums:
        dpre = dy.new_empty(d, dtype=torch.float32)
        if post_weight is not None:
            dpost = torch.empty_like(dpre)
        if gate is not None and not rows:
            dgate = torch.empty_like(dpre)
        nws = lib().moe_block_norm_grad_workspace_bytes(T, d)
        ws = dy.new_empty(nws, dtype=torch.uint8) if nws else None
    _run("moe_block_norm_grad", dev, b, dy.data_ptr(), _ptr(dh), x.data_ptr(), h.data_ptr(), T, d, dx.data_ptr(),
         dres.data_ptr(), _ptr(dpre), _ptr(dpost), _ptr(dgate), _ptr(ws), nws)
    return dx, dres, dpre, dpost, dgate


@dataclass
class W4Weights:
    """4-bit weights [N, K] in the library's layout, from w4_tile."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None
    N: int
    K: int
    group: int

    def __post_init__(self):
        # (the library goes by N, K and group: smaller tensors would be read past their ends)
        dev, shape = self.codes.get_device(), (self.N, self.K // self.group if self.group > 0 else 0)
        _arg(self.codes, "codes", (self.N, self.K // 2), (torch.uint8,), dev)
        _arg(self.scales, "scales", shape, (torch.bfloat16, torch.float16), dev)
        if self.zeros is not None:
            _arg(self.zeros, "zeros", shape, (torch.uint8,), dev)

    def struct(self, layout: int = LAYOUT_TILED) -> W4:
        fmt = SCALE_FP16 if self.scales.dtype == torch.float16 else SCALE_BF16
        return W4(_ptr(self.codes), _ptr(self.scales), _ptr(self.zeros), self.N, self.K, self.group, fmt, layout)


def w4_tile(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None) -> W4Weights:
    """4-bit weights for gemm_w4, laid out once at load time: codes uint8 [N, K/2] (0..15, the even element in
    the low half of a byte), scales bf16 or fp16 [N, K/group], zeros uint8 [N, K/group] (None: 8)."""
    N, half = _rows(codes, "codes")
    K, G = 2 * half, _rows(scales, "scales")[1]
    dev = codes.get_device()
    _arg(codes, "codes", (N, half), (torch.uint8,), dev)
    _arg(scales, "scales", (N, G), (torch.bfloat16, torch.float16), dev)
    if G < 1 or K % G:
        raise MoEError(f"scales has {G} columns, not a divisor of K = {K}")
    if zeros is not None:
        _arg(zeros, "zeros", (N, G), (torch.uint8,), dev)
    out = W4Weights(torch.empty_like(codes), torch.empty_like(scales),
                    None if zeros is None else torch.empty_like(zeros), N, K, K // G)
    src = W4Weights(codes, scales, zeros, N, K, K // G)
    _run("moe_w4_tile", dev, src.struct(LAYOUT_ROW_MAJOR), out.codes.data_ptr(), out.scales.data_ptr(),
         _ptr(out.zeros))
    return out


def gemm_w4(x: torch.Tensor, w: W4Weights, up: W4Weights | None = None):
    """bf16 [M, N] = x [M, K] w^T with 4-bit weights from w4_tile; with `up`, SiLU(x w^T) * (x up^T)."""
    M, K = _rows(x, "x")
    dev = x.get_device()
    _arg(x, "x", (M, w.K), _BF16, dev)
    for m in (w, up):
        if m is not None and m.codes.get_device() != dev:
            raise MoEError(f"w must live on GPU {dev}, not on {m.codes.device}")
    y = x.new_empty((M, w.N))
    _run("moe_gemm_w4", dev, x.data_ptr(), M, w.struct(), None if up is None else up.struct(), y.data_ptr())
    return y


class Layer:
    """The whole layer with a workspace kept between calls (no allocation per call)."""

    def __init__(self, weights: ExpertWeights, T: int, E: int, k: int, config: int = CONFIG_AUTO,
                 device=None):
        d = weights.d_model
        f = weights.gate.shape[1]
        shf = weights.sh_gate.shape[0] if weights.has_shared else 0
        self.weights = weights
        self.p = problem(T, d, f, E, k, shared_f=shf, config=config, wdtype=weights.wdtype)
        self.w = weights.struct()
        dev = device if device is not None else weights.gate.device
        # (zeroed once: the fused single-token launch keeps its counters, which every call
        # leaves zero, in the first FUSED_SYNC_BYTES)
        self.ws = torch.zeros(max(1, lib().moe_layer_workspace_bytes(ctypes.byref(self.p))),
                              dtype=torch.uint8, device=dev)
        self.out = torch.empty((T, d), dtype=torch.int16, device=dev)

    def __call__(self, logits, x, keep: dict | None = None, out=None):
        r = Routing()
        if keep:
            for name in keep:
                setattr(r, name, _ptr(keep[name]))
        out = self.out if out is None else out
        _check(lib().moe_layer(ctypes.byref(self.p), _ptr(logits), _ptr(x), ctypes.byref(self.w),
                               _ptr(out), ctypes.byref(r), _ptr(self.ws), self.ws.numel(),
                               _stream()), "moe_layer")
        return out

    def traced(self, logits, x, events, keep: dict | None = None, out=None):
        """Same as __call__, recording the TRACE_EVENTS hipEvent_t handles in `events` at the
        phase boundaries (see moe_layer_traced in the C header)."""
        r = Routing()
        if keep:
            for name in keep:
                setattr(r, name, _ptr(keep[name]))
        out = self.out if out is None else out
        arr = (ctypes.c_void_p * TRACE_EVENTS)(*events)
        _check(lib().moe_layer_traced(ctypes.byref(self.p), _ptr(logits), _ptr(x),
                                      ctypes.byref(self.w), _ptr(out), ctypes.byref(r),
                                      _ptr(self.ws), self.ws.numel(), arr, TRACE_EVENTS,
                                      _stream()), "moe_layer_traced")
        return out


def layer(logits, x, weights: ExpertWeights, k: int, config: int = CONFIG_AUTO, keep_routing=False):
    """One call of the whole layer; returns out (bf16 bits, int16) and optionally the routing."""
    T, E = logits.shape
    L = Layer(weights, T, E, k, config)
    keep = None
    if keep_routing:
        dev = logits.device
        n = T * k
        keep = dict(topk_ids=torch.empty((T, k), dtype=torch.int32, device=dev),
                    topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
                    counts=torch.empty(E, dtype=torch.int32, device=dev),
                    offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                    perm_src=torch.empty(n, dtype=torch.int32, device=dev),
                    slot_dst=torch.empty(n, dtype=torch.int32, device=dev))
    out = L(logits, x, keep)
    return (out, keep) if keep_routing else out


def layer_noalloc(logits, x, weights: ExpertWeights, k: int, out=None, config: int = CONFIG_AUTO,
                  keep: dict | None = None):
    """The whole layer on the library's static per-GPU scratch (moe_layer_noalloc): nothing is
    allocated for the call apart from `out` when the caller passes none."""
    T, E = logits.shape
    d = weights.d_model
    f = weights.gate.shape[1]
    shf = weights.sh_gate.shape[0] if weights.has_shared else 0
    p = problem(T, d, f, E, k, shared_f=shf, config=config, wdtype=weights.wdtype)
    w = weights.struct()
    if out is None:
        out = torch.empty((T, d), dtype=torch.int16, device=logits.device)
    r = Routing()
    if keep:
        for name in keep:
            setattr(r, name, _ptr(keep[name]))
    _check(lib().moe_layer_noalloc(ctypes.byref(p), _ptr(logits), _ptr(x), ctypes.byref(w),
                                   _ptr(out), ctypes.byref(r), _stream()), "moe_layer_noalloc")
    return out
