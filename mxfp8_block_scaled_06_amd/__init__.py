"""MXFP8 quantization + block-scaled grouped GEMM for MoE routed experts (gfx950).

Thin Python binding of the C ABI in include/mxmoe.h.  Every function
marshals torch tensors (device memory and the current stream) into the C
call; all arithmetic runs in the HIP kernels of libmxmoe.so.  If the library
has not been built, every entry point raises: there is no CPU fallback.

Build:  python -m mxfp8_block_scaled_06_amd.build
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

__all__ = [
    "MXError", "library_path", "load_library", "version",
    "mx_quantize_rowwise", "mx_quantize_colwise", "mx_quantize_32x32",
    "mx_grouped_gemm_mx", "mx_grouped_gemm_mx_f32", "mx_grouped_mm_workspace_bytes", "mx_scales_to_gemm_layout",
    "mx_grouped_mm_fwd", "mx_grouped_mm_dgrad", "mx_grouped_mm_wgrad",
    "mx_quantize_weights", "mx_quantize_dual", "mx_quantize_rowwise_gather",
    "mx_grouped_mm_fwd_q", "mx_grouped_mm_dgrad_q", "mx_grouped_mm", "mx_linear",
    "OP_FWD", "OP_DGRAD", "OP_WGRAD", "OP_FWD_Q", "OP_DGRAD_Q", "SCALES_ROWMAJOR", "SCALES_GEMM",
    "mx_check_offsets", "check_offsets", "mx_grouped_mm_fwd_q_noalloc", "NOALLOC_SCRATCH_BYTES",
    "mx_route", "route_capacity", "mx_quantize_dual_gather", "mx_grouped_gemm_mx_rows", "mx_routed_experts",
    "mx_topk_sum_rows", "mx_route_workspace_bytes",
    "mx_quantize_rowwise_fp4", "mx_dequantize_fp4", "mx_quantize_weights_fp4",
    "mx_grouped_gemm_mxfp4", "mx_grouped_mm_fwd_fp4", "mx_grouped_mm_dgrad_fp4", "mx_grouped_mm_fp4_workspace_bytes",
    "mx_moe_few_tokens", "mx_moe_few_tokens_workspace_bytes", "MOE_MAX_TOKENS", "MOE_MAX_TOPK",
    "mx_dequantize", "mx_topk_router", "mx_topk_router_fwd", "mx_topk_router_bwd", "ROUTER_MAX_GROUPS",
    "mx_swiglu", "mx_swiglu_fwd", "mx_swiglu_bwd", "mx_swiglu_quantize", "mx_swiglu_quantize_fwd",
    "mx_swiglu_quantize_bwd", "mx_swiglu_quantize_workspace_bytes",
    "mx_topk_combine", "mx_topk_combine_fwd", "mx_topk_combine_bwd", "mx_moe_layer",
]

OP_FWD, OP_DGRAD, OP_WGRAD, OP_FWD_Q, OP_DGRAD_Q = 0, 1, 2, 3, 4
SCALES_ROWMAJOR, SCALES_GEMM = 0, 1
_LAYOUTS = {"rowmajor": SCALES_ROWMAJOR, "gemm": SCALES_GEMM}
MOE_MAX_TOKENS, MOE_MAX_TOPK = 128, 32     # MX_MOE_MAX_TOKENS, MX_MOE_MAX_TOPK
FORMATS = {"mxfp8": 0, "mxfp4": 1}    # MX_FMT_FP8, MX_FMT_FP4
SCORES = {"softmax": 0, "sigmoid": 1}     # MX_SCORE_SOFTMAX, MX_SCORE_SIGMOID
GROUP_SCORES = {"max": 0, "top2": 1}      # MX_GROUP_MAX, MX_GROUP_TOP2
ROUTER_MAX_GROUPS = 64                    # MX_ROUTER_MAX_GROUPS
OFFS_DECREASING, OFFS_RANGE, OFFS_LAST, OFFS_ALIGN = 1, 2, 4, 8
NOALLOC_SCRATCH_BYTES = 128 << 20     # MX_NOALLOC_SCRATCH_BYTES of include/mxmoe.h
_STATUS = {0: "MX_OK", 1: "MX_ERR_NULL", 2: "MX_ERR_SHAPE", 3: "MX_ERR_ALIGN", 4: "MX_ERR_WORKSPACE",
           5: "MX_ERR_HIP", 6: "MX_ERR_LAYOUT"}

_PKG = os.path.dirname(os.path.abspath(__file__))
_lib = None


class MXError(RuntimeError):
    """A C-ABI call returned a status other than MX_OK."""

    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {text}")
        self.status = status


def library_path() -> str:
    return os.path.join(_PKG, "libmxmoe.so")


def load_library():
    """Load libmxmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m mxfp8_block_scaled_06_amd.build`")
    lib = ctypes.CDLL(path)
    c_i64, c_vp, c_int, c_sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.mx_last_error.restype = ctypes.c_char_p
    lib.mx_version.restype = ctypes.c_char_p
    for name in ("mx_quantize_rowwise", "mx_quantize_colwise", "mx_quantize_32x32"):
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp]
    for name in ("mx_grouped_gemm_mx", "mx_grouped_gemm_mx_f32"):
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = [c_vp, c_vp, c_vp, c_vp, c_int, c_vp, c_int, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp]
    lib.mx_grouped_gemm_mx_ordered.restype = c_int
    lib.mx_grouped_gemm_mx_ordered.argtypes = [c_vp, c_vp, c_vp, c_vp, c_int, c_vp, c_int, c_i64, c_i64, c_i64, c_i64,
                                               c_vp, ctypes.c_uint64, c_vp]
    lib.mx_grouped_gemm_mx_rows.restype = c_int
    lib.mx_grouped_gemm_mx_rows.argtypes = [c_vp, c_vp, c_vp, c_vp, c_int, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp,
                                            c_vp, c_i64, c_vp]
    lib.mx_grouped_gemm_mx_rows_f32.restype = c_int
    lib.mx_grouped_gemm_mx_rows_f32.argtypes = lib.mx_grouped_gemm_mx_rows.argtypes
    lib.mx_topk_sum_rows.restype = c_int
    lib.mx_topk_sum_rows.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]
    lib.mx_route.restype = c_int
    lib.mx_route.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
    lib.mx_route_workspace_bytes.restype = c_sz
    lib.mx_route_workspace_bytes.argtypes = [c_i64, c_i64]
    lib.mx_quantize_dual_gather.restype = c_int
    lib.mx_quantize_dual_gather.argtypes = [c_vp, c_i64, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp,
                                            c_vp]
    lib.mx_check_offsets.restype = c_int
    lib.mx_check_offsets.argtypes = [c_vp, c_i64, c_i64, ctypes.c_int32, c_vp, c_vp]
    lib.mx_scales_to_gemm_layout.restype = c_int
    lib.mx_scales_to_gemm_layout.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]
    lib.mx_grouped_mm_workspace_bytes.restype = c_sz
    lib.mx_grouped_mm_workspace_bytes.argtypes = [c_int, c_i64, c_i64, c_i64, c_i64]
    for name in ("mx_grouped_mm_fwd", "mx_grouped_mm_dgrad", "mx_grouped_mm_wgrad"):
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_sz, c_vp]
    lib.mx_quantize_rowwise_gather.restype = c_int
    lib.mx_quantize_rowwise_gather.argtypes = [c_vp, c_i64, c_vp, c_i64, c_i64, c_vp, c_vp, c_vp]
    lib.mx_quantize_weights.restype = c_int
    lib.mx_quantize_weights.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp]
    lib.mx_quantize_dual.restype = c_int
    lib.mx_quantize_dual.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp]
    for name in ("mx_grouped_mm_fwd_q", "mx_grouped_mm_dgrad_q"):
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_sz, c_vp]
    lib.mx_grouped_mm_fwd_q_noalloc.restype = c_int
    lib.mx_grouped_mm_fwd_q_noalloc.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp]
    lib.mx_quantize_rowwise_fp4.restype = c_int
    lib.mx_quantize_rowwise_fp4.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_int, c_vp]
    lib.mx_dequantize_fp4.restype = c_int
    lib.mx_dequantize_fp4.argtypes = [c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_vp, c_vp]
    lib.mx_quantize_weights_fp4.restype = c_int
    lib.mx_quantize_weights_fp4.argtypes = lib.mx_quantize_weights.argtypes
    lib.mx_grouped_gemm_mxfp4.restype = c_int
    lib.mx_grouped_gemm_mxfp4.argtypes = [c_vp, c_vp, c_int, c_vp, c_vp, c_int, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp,
                                          c_i64, c_vp, c_int, c_vp]
    lib.mx_grouped_mm_fp4_workspace_bytes.restype = c_sz
    lib.mx_grouped_mm_fp4_workspace_bytes.argtypes = [c_i64, c_i64, c_int]
    for name in ("mx_grouped_mm_fwd_fp4", "mx_grouped_mm_dgrad_fp4"):
        f = getattr(lib, name)
        f.restype = c_int
        f.argtypes = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_int, c_vp, c_vp, c_sz, c_vp]
    lib.mx_moe_few_tokens_workspace_bytes.restype = c_sz
    lib.mx_moe_few_tokens_workspace_bytes.argtypes = [c_i64, c_i64, c_i64]
    lib.mx_moe_few_tokens.restype = c_int
    lib.mx_moe_few_tokens.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_int, c_i64, c_i64, c_i64, c_i64,
                                      c_i64, c_vp, c_vp, c_vp, c_sz, c_vp]
    c_f = ctypes.c_float
    lib.mx_dequantize.restype = c_int
    lib.mx_dequantize.argtypes = lib.mx_dequantize_fp4.argtypes
    lib.mx_topk_router_fwd.restype = c_int
    lib.mx_topk_router_fwd.argtypes = [c_vp, c_int, c_vp, c_i64, c_i64, c_i64, c_int, c_i64, c_i64, c_int, c_int, c_f,
                                       c_vp, c_vp, c_vp]
    lib.mx_topk_router_bwd.restype = c_int
    lib.mx_topk_router_bwd.argtypes = [c_vp, c_int, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int, c_int, c_f, c_vp, c_vp]
    lib.mx_swiglu_fwd.restype = c_int
    lib.mx_swiglu_fwd.argtypes = [c_vp, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp]
    lib.mx_swiglu_bwd.restype = c_int
    lib.mx_swiglu_bwd.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_vp, c_vp]
    lib.mx_swiglu_quantize.restype = c_int
    lib.mx_swiglu_quantize.argtypes = [c_vp, c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp]
    lib.mx_swiglu_quantize_fwd.restype = c_int
    lib.mx_swiglu_quantize_fwd.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp,
                                           c_vp, c_vp]
    lib.mx_swiglu_quantize_workspace_bytes.restype = c_sz
    lib.mx_swiglu_quantize_workspace_bytes.argtypes = [c_i64, c_i64]
    lib.mx_swiglu_quantize_bwd.restype = c_int
    lib.mx_swiglu_quantize_bwd.argtypes = [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp,
                                           c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
    lib.mx_topk_combine_fwd.restype = c_int
    lib.mx_topk_combine_fwd.argtypes = [c_vp, c_int, c_vp, c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]
    lib.mx_topk_combine_bwd.restype = c_int
    lib.mx_topk_combine_bwd.argtypes = [c_vp, c_int, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp]
    _lib = lib
    return lib


_bound = None


def _native():
    """_nodes.so (csrc/mx_nodes.cpp): autograd nodes, and calls that allocate their results; each returns None
    where an operand does not fit, for the checks here to say which."""
    global _bound
    if _bound is None:
        load_library()
        try:
            from . import _nodes as nodes
        except ImportError as e:
            raise RuntimeError(f"_nodes.so is missing or does not fit this torch ({e}): build it with "
                               "`python -m mxfp8_block_scaled_06_amd.build`") from e
        nodes.set_error(MXError)
        _bound = nodes
    return _bound


def version() -> str:
    return load_library().mx_version().decode()


def _check(fn: str, status: int):
    if status != 0:
        raise MXError(fn, status, load_library().mx_last_error().decode())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    import torch
    # the raw handle alone where torch offers it: 0.1 us against 1.9 for a Stream object
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _require(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, shape, dtype, device, name):
    """An output buffer: allocated when None, else checked to be exactly what
    the kernel writes (the C ABI sees only a pointer and cannot)."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    shape = tuple(map(int, shape))
    if isinstance(t, torch.Tensor) and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    _require(t, dtype, name)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _as3d(x):
    shape = tuple(x.shape)
    if len(shape) == 2:
        return 1, *shape
    if len(shape) == 3:
        return shape
    raise ValueError("expected a 2-D or 3-D tensor")


# ---------------------------------------------------------------------------
# Quantizers
# ---------------------------------------------------------------------------
def mx_quantize_rowwise(x, q=None, s=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """1x32 blocks along the last axis.  x bf16 [..., R, C] -> (q uint8 same shape, s uint8 [..., R, C/32])."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    B, R, C = _as3d(x)
    lead = x.shape[:-1]
    q = _out(q, x.shape, torch.uint8, x.device, "q")
    s = _out(s, (*lead, C // 32 if C % 32 == 0 else 0), torch.uint8, x.device, "s")
    _check("mx_quantize_rowwise", lib.mx_quantize_rowwise(_ptr(x), B, R, C, _ptr(q), _ptr(s), _stream(x.device)))
    return q, s


def mx_quantize_colwise(x, q_t=None, s_t=None):
    """32x1 blocks along rows, output transposed.  x bf16 [B?, R, C] ->
    (q_t uint8 [B?, C, R], s_t uint8 [B?, C, R/32])."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    B, R, C = _as3d(x)
    lead = x.shape[:-2]
    q_t = _out(q_t, (*lead, C, R), torch.uint8, x.device, "q_t")
    s_t = _out(s_t, (*lead, C, R // 32 if R % 32 == 0 else 0), torch.uint8, x.device, "s_t")
    _check("mx_quantize_colwise",
           lib.mx_quantize_colwise(_ptr(x), B, R, C, _ptr(q_t), _ptr(s_t), _stream(x.device)))
    return q_t, s_t


def mx_quantize_32x32(x, q=None, s=None):
    """32x32 blocks.  x bf16 [B?, R, C] -> (q uint8 same shape, s uint8 [B?, R/32, C/32])."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    B, R, C = _as3d(x)
    lead = x.shape[:-2]
    q = _out(q, x.shape, torch.uint8, x.device, "q")
    s = _out(s, (*lead, R // 32, C // 32), torch.uint8, x.device, "s")
    _check("mx_quantize_32x32", lib.mx_quantize_32x32(_ptr(x), B, R, C, _ptr(q), _ptr(s), _stream(x.device)))
    return q, s


def mx_scales_to_gemm_layout(s, out=None):
    """Row-major scales [B?, R, KB] -> the GEMM's blocked layout [B?, KB/4, R, 4]."""
    import torch
    lib = load_library()
    _require(s, torch.uint8, "s")
    B, R, KB = _as3d(s)
    out = _out(out, (*s.shape[:-2], KB // 4, R, 4), torch.uint8, s.device, "out")
    _check("mx_scales_to_gemm_layout",
           lib.mx_scales_to_gemm_layout(_ptr(s), B, R, KB, _ptr(out), _stream(s.device)))
    return out


# ---------------------------------------------------------------------------
# Grouped GEMM on prequantized operands
# ---------------------------------------------------------------------------
def mx_grouped_gemm_mx(X, sX, Y, sY, offs, mode: int, out=None, out_dtype=None, scale_layout: str = "gemm"):
    """C[i,j] = sum_k X[i,k] Y[j,k] 2^(sX+sY-254).  mode 0: Y [E,J,Kc], C [I,J];
    mode 1 (groups over k): Y [J,Kc], C [E,I,J].  The scales must be in the
    GEMM's blocked layout (what mx_quantize_weights / mx_quantize_dual write,
    or mx_scales_to_gemm_layout of a quantizer's row-major scales):
    sX [Kc/128, I, 4]; sY [E, Kc/128, J, 4] in mode 0, [Kc/128, J, 4] in mode 1.
    Row-major scales raise (their shapes differ).  Returns C (bf16, or fp32
    with out_dtype=torch.float32)."""
    import torch
    lib = load_library()
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    I, J, Kc, E, layout = _gemm_operands(X, sX, Y, sY, offs, mode, scale_layout)
    out = _out(out, (I, J) if mode == 0 else (E, I, J), out_dtype, X.device, "out")
    name = "mx_grouped_gemm_mx" if out_dtype == torch.bfloat16 else "mx_grouped_gemm_mx_f32"
    _check(name, getattr(lib, name)(_ptr(X), _ptr(sX), _ptr(Y), _ptr(sY), layout, _ptr(offs), mode, I, J, Kc, E,
                                    _ptr(out), _stream(X.device)))
    return out


def _gemm_operands(X, sX, Y, sY, offs, mode, scale_layout):
    """Shape checks of the GEMM operands; returns (I, J, Kc, E, layout code)."""
    import torch
    if scale_layout not in ("gemm", "rowmajor"):
        raise ValueError("scale_layout must be 'gemm' or 'rowmajor'")
    for t, n in ((X, "X"), (sX, "sX"), (Y, "Y"), (sY, "sY")):
        _require(t, torch.uint8, n)
    _require(offs, torch.int32, "offs")
    E = offs.shape[0]
    if X.dim() != 2:
        raise ValueError("X must be [I, Kc]")
    I, Kc = X.shape
    if mode == 0:
        if Y.dim() != 3 or Y.shape[0] != E or Y.shape[2] != Kc:
            raise ValueError(f"mode 0: Y must be [E={E}, J, Kc={Kc}], got {tuple(Y.shape)}")
        J = Y.shape[1]
    else:
        if Y.dim() != 2 or Y.shape[1] != Kc:
            raise ValueError(f"mode 1: Y must be [J, Kc={Kc}], got {tuple(Y.shape)}")
        J = Y.shape[0]
    if scale_layout == "gemm":
        want_x = (Kc // 128, I, 4)
        want_y = (E, Kc // 128, J, 4) if mode == 0 else (Kc // 128, J, 4)
        for t, want, n in ((sX, want_x, "sX"), (sY, want_y, "sY")):
            if tuple(t.shape) != want:
                hint = (" (these are row-major scales: convert them with mx_scales_to_gemm_layout)"
                        if t.dim() == len(want) - 1 and t.shape[-1] == Kc // 32 else "")
                raise ValueError(f"{n} must be in the GEMM scale layout {want}, got {tuple(t.shape)}{hint}")
    return I, J, Kc, E, SCALES_GEMM if scale_layout == "gemm" else SCALES_ROWMAJOR


def mx_grouped_gemm_mx_rows(X, sX, Y, sY, offs, row_map, c_rows: Optional[int] = None, out=None,
                            out_dtype=None):
    """mx_grouped_gemm_mx (mode 0) storing grouped row i to out row
    row_map[i] (rows whose entry lies outside [0, c_rows) are dropped; out
    rows no entry names are left as they were).  row_map int32 [I] on the GPU
    (the `rows` of mx_route); out bf16 (or fp32 with out_dtype=torch.float32)
    [c_rows, J] (default c_rows: out's rows, else I; a new out starts at
    zero)."""
    import torch
    lib = load_library()
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    I, J, Kc, E, layout = _gemm_operands(X, sX, Y, sY, offs, 0, "gemm")
    _require(row_map, torch.int32, "row_map")
    if tuple(row_map.shape) != (I,):
        raise ValueError(f"row_map must be int32 [{I}] (one entry per row of X), got {tuple(row_map.shape)}")
    if c_rows is None:
        c_rows = out.shape[0] if out is not None else I
    if out is None:
        out = torch.zeros((c_rows, J), dtype=out_dtype, device=X.device)
    out = _out(out, (c_rows, J), out_dtype, X.device, "out")
    name = "mx_grouped_gemm_mx_rows" if out_dtype == torch.bfloat16 else "mx_grouped_gemm_mx_rows_f32"
    _check(name, getattr(lib, name)(_ptr(X), _ptr(sX), _ptr(Y), _ptr(sY), layout, _ptr(offs), I, J, Kc, E,
                                    _ptr(row_map), _ptr(out), int(c_rows), _stream(X.device)))
    return out


def mx_topk_sum_rows(x, k: int, out=None):
    """x fp32 [T*k, cols] -> bf16 [T, cols]: each token's k rows summed in fp32
    in slot order, rounded to nearest even once (the top-k gather's gradient)."""
    import torch
    lib = load_library()
    _require(x, torch.float32, "x")
    if x.dim() != 2 or x.shape[0] % k:
        raise ValueError(f"x must be [T*k, cols] with k={k}, got {tuple(x.shape)}")
    T, cols = x.shape[0] // k, x.shape[1]
    out = _out(out, (T, cols), torch.bfloat16, x.device, "out")
    _check("mx_topk_sum_rows", lib.mx_topk_sum_rows(_ptr(x), T, int(k), cols, _ptr(out), _stream(x.device)))
    return out


def mx_grouped_gemm_mx_ordered(X, sX, Y, sY, offs, mode: int, order_seed: int, out=None):
    """mx_grouped_gemm_mx (bf16) with workgroups dealt to tiles in a seeded
    pseudo-random order (race checks: the result must not depend on it)."""
    import torch
    lib = load_library()
    I, J, Kc, E, layout = _gemm_operands(X, sX, Y, sY, offs, mode, "gemm")
    out = _out(out, (I, J) if mode == 0 else (E, I, J), torch.bfloat16, X.device, "out")
    _check("mx_grouped_gemm_mx_ordered",
           lib.mx_grouped_gemm_mx_ordered(_ptr(X), _ptr(sX), _ptr(Y), _ptr(sY), layout, _ptr(offs), mode, I, J, Kc, E,
                                          _ptr(out), int(order_seed), _stream(X.device)))
    return out


def mx_grouped_gemm_mx_f32(X, sX, Y, sY, offs, mode: int, out=None):
    """mx_grouped_gemm_mx with fp32 output (accumulators stored unrounded)."""
    import torch
    return mx_grouped_gemm_mx(X, sX, Y, sY, offs, mode, out=out, out_dtype=torch.float32)


def mx_grouped_mm_workspace_bytes(op: int, M: int, N: int, K: int, E: int) -> int:
    return int(load_library().mx_grouped_mm_workspace_bytes(op, M, N, K, E))


def _offs(offs, E):
    """offs: int32 [E] group END offsets on the GPU (the kernels read E entries)."""
    import torch
    if isinstance(offs, torch.Tensor) and (offs.dim() != 1 or offs.shape[0] != E):
        raise ValueError(f"offs must be int32 [{E}] (one END offset per expert), got {tuple(offs.shape)}")
    _require(offs, torch.int32, "offs")


def _ws(op, M, N, K, E, device, ws):
    import torch
    need = mx_grouped_mm_workspace_bytes(op, M, N, K, E)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return ws


# ---------------------------------------------------------------------------
# Grouped GEMMs on bf16 inputs (quantize both operands, then GEMM)
# ---------------------------------------------------------------------------
def mx_grouped_mm_fwd(A, W, offs, out=None, ws=None):
    """out [M, N] = A [M, K] @ W[e] [N, K]^T per expert group (offs: int32 END offsets)."""
    import torch
    lib = load_library()
    _require(A, torch.bfloat16, "A")
    _require(W, torch.bfloat16, "W")
    _require(offs, torch.int32, "offs")
    M, K = A.shape
    E, N, K2 = W.shape
    if K2 != K:
        raise ValueError(f"A has K={K} but W has K={K2}")
    _offs(offs, E)
    out = _out(out, (M, N), torch.bfloat16, A.device, "out")
    ws = _ws(OP_FWD, M, N, K, E, A.device, ws)
    _check("mx_grouped_mm_fwd",
           lib.mx_grouped_mm_fwd(_ptr(A), _ptr(W), _ptr(offs), M, N, K, E, _ptr(out), _ptr(ws), ws.numel(),
                                 _stream(A.device)))
    return out


def mx_grouped_mm_dgrad(dOut, W, offs, out=None, ws=None):
    """dA [M, K] = dOut [M, N] @ W[e] [N, K] per expert group."""
    import torch
    lib = load_library()
    _require(dOut, torch.bfloat16, "dOut")
    _require(W, torch.bfloat16, "W")
    _require(offs, torch.int32, "offs")
    M, N = dOut.shape
    E, N2, K = W.shape
    if N2 != N:
        raise ValueError(f"dOut has N={N} but W has N={N2}")
    _offs(offs, E)
    out = _out(out, (M, K), torch.bfloat16, dOut.device, "out")
    ws = _ws(OP_DGRAD, M, N, K, E, dOut.device, ws)
    _check("mx_grouped_mm_dgrad",
           lib.mx_grouped_mm_dgrad(_ptr(dOut), _ptr(W), _ptr(offs), M, N, K, E, _ptr(out), _ptr(ws), ws.numel(),
                                   _stream(dOut.device)))
    return out


def mx_grouped_mm_wgrad(dOut, A, offs, out=None, ws=None):
    """dW [E, N, K], dW[e] = dOut[g_e]^T @ A[g_e] (groups padded to multiples of 32)."""
    import torch
    lib = load_library()
    _require(dOut, torch.bfloat16, "dOut")
    _require(A, torch.bfloat16, "A")
    _require(offs, torch.int32, "offs")
    M, N = dOut.shape
    M2, K = A.shape
    if M2 != M:
        raise ValueError(f"dOut has M={M} but A has M={M2}")
    E = offs.shape[0]
    out = _out(out, (E, N, K), torch.bfloat16, A.device, "out")
    ws = _ws(OP_WGRAD, M, N, K, E, A.device, ws)
    _check("mx_grouped_mm_wgrad",
           lib.mx_grouped_mm_wgrad(_ptr(dOut), _ptr(A), _ptr(offs), M, N, K, E, _ptr(out), _ptr(ws), ws.numel(),
                                   _stream(A.device)))
    return out


# ---------------------------------------------------------------------------
# Prequantized expert weights (both orientations in one pass)
# ---------------------------------------------------------------------------
def mx_quantize_weights(W, q=None, s=None, q_t=None, s_t=None):
    """W bf16 [E, N, K] -> (q [E, N, K], s [E, K/128, N, 4], q_t [E, K, N], s_t [E, N/128, K, 4]):
    rowwise codes along K and colwise codes along N (stored transposed), scales
    in the GEMM layout.  N and K must be multiples of 128."""
    import torch
    lib = load_library()
    _require(W, torch.bfloat16, "W")
    if W.dim() != 3:
        raise ValueError("W must be [E, N, K]")
    E, N, K = W.shape
    dev = W.device
    q = _out(q, (E, N, K), torch.uint8, dev, "q")
    s = _out(s, (E, K // 128, N, 4), torch.uint8, dev, "s")
    q_t = _out(q_t, (E, K, N), torch.uint8, dev, "q_t")
    s_t = _out(s_t, (E, N // 128, K, 4), torch.uint8, dev, "s_t")
    _check("mx_quantize_weights", lib.mx_quantize_weights(_ptr(W), E, N, K, _ptr(q), _ptr(s), _ptr(q_t), _ptr(s_t),
                                                          _stream(dev)))
    return q, s, q_t, s_t


def mx_quantize_dual(x, ldq: Optional[int] = None, q=None, s=None, q_t=None, s_t=None):
    """Activations x bf16 [rows, cols] in both orientations from one read:
    (q [rows, cols], s [cols/128, rows, 4]) = X of the rows-grouped GEMM, and
    (q_t [cols, ldq], s_t [ldq/128, cols, 4]) = a wgrad operand with Kc = ldq
    (default: rows rounded up to 128; the padding columns are zero codes)."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    rows, cols = x.shape
    if ldq is None:
        ldq = (rows + 127) // 128 * 128
    dev = x.device
    q = _out(q, (rows, cols), torch.uint8, dev, "q")
    s = _out(s, (cols // 128, rows, 4), torch.uint8, dev, "s")
    q_t = _out(q_t, (cols, ldq), torch.uint8, dev, "q_t")
    s_t = _out(s_t, (ldq // 128, cols, 4), torch.uint8, dev, "s_t")
    _check("mx_quantize_dual", lib.mx_quantize_dual(_ptr(x), rows, cols, ldq, _ptr(q), _ptr(s), _ptr(q_t), _ptr(s_t),
                                                    _stream(dev)))
    return q, s, q_t, s_t


def mx_grouped_mm_fwd_q(A, qW, sW, offs, out=None, ws=None):
    """mx_grouped_mm_fwd with W given as (q, s) of mx_quantize_weights."""
    import torch
    lib = load_library()
    _require(A, torch.bfloat16, "A")
    _require(qW, torch.uint8, "qW")
    _require(sW, torch.uint8, "sW")
    _require(offs, torch.int32, "offs")
    M, K = A.shape
    E, N, K2 = qW.shape
    if K2 != K:
        raise ValueError(f"A has K={K} but qW has K={K2}")
    _offs(offs, E)
    if sW.numel() != E * N * (K // 32):
        raise ValueError(f"sW must hold E*N*K/32 = {E * N * (K // 32)} bytes, got {sW.numel()}")
    out = _out(out, (M, N), torch.bfloat16, A.device, "out")
    ws = _ws(OP_FWD_Q, M, N, K, E, A.device, ws)
    _check("mx_grouped_mm_fwd_q",
           lib.mx_grouped_mm_fwd_q(_ptr(A), _ptr(qW), _ptr(sW), _ptr(offs), M, N, K, E, _ptr(out), _ptr(ws),
                                   ws.numel(), _stream(A.device)))
    return out


def mx_grouped_mm_dgrad_q(dOut, qWt, sWt, offs, out=None, ws=None):
    """mx_grouped_mm_dgrad with W given as (q_t, s_t) of mx_quantize_weights."""
    import torch
    lib = load_library()
    _require(dOut, torch.bfloat16, "dOut")
    _require(qWt, torch.uint8, "qWt")
    _require(sWt, torch.uint8, "sWt")
    _require(offs, torch.int32, "offs")
    M, N = dOut.shape
    E, K, N2 = qWt.shape
    if N2 != N:
        raise ValueError(f"dOut has N={N} but qWt has N={N2}")
    _offs(offs, E)
    if sWt.numel() != E * K * (N // 32):
        raise ValueError(f"sWt must hold E*K*N/32 = {E * K * (N // 32)} bytes, got {sWt.numel()}")
    out = _out(out, (M, K), torch.bfloat16, dOut.device, "out")
    ws = _ws(OP_DGRAD_Q, M, N, K, E, dOut.device, ws)
    _check("mx_grouped_mm_dgrad_q",
           lib.mx_grouped_mm_dgrad_q(_ptr(dOut), _ptr(qWt), _ptr(sWt), _ptr(offs), M, N, K, E, _ptr(out), _ptr(ws),
                                     ws.numel(), _stream(dOut.device)))
    return out


def mx_check_offsets(offs, M: int, align: int = 1, status=None):
    """Validity bitmask of the group offsets, computed on the device into
    `status` (int32 [1] on the GPU; returned without synchronizing).  0 = valid;
    OFFS_DECREASING / OFFS_RANGE / OFFS_LAST / OFFS_ALIGN otherwise."""
    import torch
    lib = load_library()
    _require(offs, torch.int32, "offs")
    if offs.dim() != 1:
        raise ValueError("offs must be int32 [E]")
    status = _out(status, (1,), torch.int32, offs.device, "status")
    _check("mx_check_offsets", lib.mx_check_offsets(_ptr(offs), offs.shape[0], int(M), int(align), _ptr(status),
                                                    _stream(offs.device)))
    return status


def check_offsets(offs, M: int, align: int = 1):
    """Raise ValueError, naming every violated rule, unless the group offsets
    are valid (reads the device status word: one synchronization)."""
    bits = int(mx_check_offsets(offs, M, align).item())
    if bits:
        why = [text for bit, text in ((OFFS_DECREASING, "an offset is below its predecessor"),
                                      (OFFS_RANGE, f"an offset lies outside [0, {M}]"),
                                      (OFFS_LAST, f"the last offset is not M={M}"),
                                      (OFFS_ALIGN, f"a group starts off a multiple of {align} (pad every group "
                                                   f"with zero rows to a multiple of {align})")) if bits & bit]
        raise ValueError("invalid group offsets: " + "; ".join(why))


def mx_grouped_mm_fwd_q_noalloc(A, qW, sW, offs, out):
    """mx_grouped_mm_fwd_q without a workspace: the library quantizes A into a
    static device array (NOALLOC_SCRATCH_BYTES) instead, so nothing is
    allocated (for graph capture or loops that cannot allocate).  `out` bf16
    [M, N] is the caller's.  Calls overlapping on one GPU share the array and
    race."""
    import torch
    lib = load_library()
    _require(A, torch.bfloat16, "A")
    _require(qW, torch.uint8, "qW")
    _require(sW, torch.uint8, "sW")
    _require(offs, torch.int32, "offs")
    M, K = A.shape
    E, N, K2 = qW.shape
    if K2 != K:
        raise ValueError(f"A has K={K} but qW has K={K2}")
    _offs(offs, E)
    if tuple(sW.shape) != (E, K // 128, N, 4):
        raise ValueError(f"sW must be in the GEMM scale layout {(E, K // 128, N, 4)}, got {tuple(sW.shape)}")
    if out is None:
        raise ValueError("out must be given: this entry point allocates nothing")
    out = _out(out, (M, N), torch.bfloat16, A.device, "out")
    _check("mx_grouped_mm_fwd_q_noalloc",
           lib.mx_grouped_mm_fwd_q_noalloc(_ptr(A), _ptr(qW), _ptr(sW), _ptr(offs), M, N, K, E, _ptr(out),
                                           _stream(A.device)))
    return out


def mx_grouped_mm(A, W, offs, check_offsets: bool = True, weights=None, cache=None, weight_format: str = "mxfp8"):
    """Differentiable MXFP8 grouped GEMM (forward, dgrad, wgrad in the library's kernels);
    expert weights quantized once and cached across micro-batches until they change.
    weight_format="mxfp4": 4-bit weights, quantized in every call unless `weights` or a `cache` is given."""
    from .autograd import mx_grouped_mm as _f
    return _f(A, W, offs, check_offsets, weights, cache, weight_format)


def mx_linear(x, weight, weight_format: str = "mxfp8"):
    """Differentiable dense MXFP8 linear y = x @ weight^T (one expert of mx_grouped_mm)."""
    from .autograd import mx_linear as _f
    return _f(x, weight, weight_format)


def mx_quantize_rowwise_gather(x, rows, q=None, s=None):
    """Rowwise MX quantization of x[rows[r]] (rows int32 [M]; a negative index gives a zero row).
    Returns (q uint8 [M, cols], s uint8 [cols/128, M, 4] in the GEMM scale layout)."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    _require(rows, torch.int32, "rows")
    src_rows, cols = x.shape
    M = rows.shape[0]
    q = _out(q, (M, cols), torch.uint8, x.device, "q")
    s = _out(s, (cols // 128, M, 4), torch.uint8, x.device, "s")
    _check("mx_quantize_rowwise_gather",
           lib.mx_quantize_rowwise_gather(_ptr(x), src_rows, _ptr(rows), M, cols, _ptr(q), _ptr(s), _stream(x.device)))
    return q, s


# ---------------------------------------------------------------------------
# Routed experts: grouping, gather and scatter on the device
# ---------------------------------------------------------------------------
def route_capacity(n: int, E: int) -> int:
    """Rows of the grouped operands for n routed items over E experts: the
    most the groups can take once each is padded to 32 rows (n + 31 E),
    rounded up to 128 so the rows also serve as the wgrad contraction."""
    return (int(n) + 31 * int(E) + 127) // 128 * 128


def mx_route(expert_idx, E: int, cap: Optional[int] = None, offs=None, rows=None, pos=None, status=None, ws=None):
    """Group routed items by expert on the device.  expert_idx int32 [n] (a
    top-k router's [T, k] ids flattened token-major).  Returns (offs int32 [E]
    padded END offsets, rows int32 [cap] grouped row -> item or -1, pos int32
    [n] item -> grouped row, status int32 [1]: 1 if an id lies outside
    [0, E)).  `ws`: uint8 scratch of mx_route_workspace_bytes(n, E) bytes
    (allocated when None).  Nothing is synchronized."""
    import torch
    lib = load_library()
    _require(expert_idx, torch.int32, "expert_idx")
    if expert_idx.dim() != 1:
        raise ValueError("expert_idx must be int32 [n] (flatten a [T, k] router output)")
    n = expert_idx.shape[0]
    if cap is None:
        cap = route_capacity(n, E)
    dev = expert_idx.device
    offs = _out(offs, (E,), torch.int32, dev, "offs")
    rows = _out(rows, (cap,), torch.int32, dev, "rows")
    pos = _out(pos, (n,), torch.int32, dev, "pos")
    status = _out(status, (1,), torch.int32, dev, "status")
    need = mx_route_workspace_bytes(n, E)
    if ws is None:
        ws = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    _require(ws, torch.uint8, "ws")
    _check("mx_route", lib.mx_route(_ptr(expert_idx), n, int(E), int(cap), _ptr(offs), _ptr(rows), _ptr(pos),
                                    _ptr(status), _ptr(ws), ws.numel(), _stream(dev)))
    return offs, rows, pos, status


def mx_route_workspace_bytes(n: int, E: int) -> int:
    return int(load_library().mx_route_workspace_bytes(int(n), int(E)))


def mx_quantize_dual_gather(x, rows, topk: int = 1, ldq: Optional[int] = None, q=None, s=None, q_t=None, s_t=None):
    """mx_quantize_dual of the gathered rows x[rows[r] // topk] (zero rows
    where rows[r] < 0 or >= x.shape[0] * topk).  rows int32 [M] (M % 32 == 0).
    Returns (q [M, cols], s [cols/128, M, 4], q_t [cols, ldq], s_t
    [ldq/128, cols, 4]); ldq defaults to M rounded up to 128."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    _require(rows, torch.int32, "rows")
    if x.dim() != 2 or rows.dim() != 1:
        raise ValueError("x must be [src_rows, cols] and rows int32 [M]")
    src_rows, cols = x.shape
    M = rows.shape[0]
    if ldq is None:
        ldq = (M + 127) // 128 * 128
    dev = x.device
    q = _out(q, (M, cols), torch.uint8, dev, "q")
    s = _out(s, (cols // 128, M, 4), torch.uint8, dev, "s")
    q_t = _out(q_t, (cols, ldq), torch.uint8, dev, "q_t")
    s_t = _out(s_t, (ldq // 128, cols, 4), torch.uint8, dev, "s_t")
    _check("mx_quantize_dual_gather",
           lib.mx_quantize_dual_gather(_ptr(x), src_rows, _ptr(rows), int(topk), M, cols, int(ldq), _ptr(q), _ptr(s),
                                       _ptr(q_t), _ptr(s_t), _stream(dev)))
    return q, s, q_t, s_t


def mx_routed_experts(x, expert_idx, W, check: bool = True, weights=None, cache=None, weight_format: str = "mxfp8"):
    """Differentiable routed experts: out[t] = x[t] @ W[expert_idx[t]]^T for a
    top-1 router (expert_idx [T]), out[t, j] = x[t] @ W[expert_idx[t, j]]^T for
    a top-k router (expert_idx [T, k]), with the grouping, the token gather
    (inside the quantizer) and the scatter back to item order (inside the GEMM
    epilogue) on the device."""
    from .autograd import mx_routed_experts as _f
    return _f(x, expert_idx, W, check, weights, cache, weight_format)


# ---------------------------------------------------------------------------
# MXFP4 (4-bit E2M1 elements, two to a byte, E8M0 scales per 32)
# ---------------------------------------------------------------------------
def _scale_shape(scale_layout, lead, R, C):
    """Shape of the scales of [*lead, R, C] values in a layout, and its code."""
    if scale_layout == "rowmajor":
        if C % 32:
            raise ValueError(f"the last axis ({C}) must be a multiple of 32")
        return (*lead, R, C // 32), SCALES_ROWMAJOR
    if scale_layout == "gemm":
        if C % 128:
            raise ValueError(f"the last axis ({C}) must be a multiple of 128 for scales in the GEMM layout")
        return (*lead, C // 128, R, 4), SCALES_GEMM
    raise ValueError("scale_layout must be 'gemm' or 'rowmajor'")


_CURRENT = contextlib.nullcontext()


def _on(device):
    """Makes `device` the current one for a launch; no cost where it is (nothing
    to do for the CPU, whose tensors the calls refuse)."""
    import torch
    if device.type != "cuda" or device.index == torch.cuda.current_device():
        return _CURRENT
    return torch.cuda.device(device)


def _same_device(first, *rest):
    """Every tensor on the device of the first one (the kernels run there)."""
    dev = first.device
    for t in rest:
        if t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")


def mx_quantize_rowwise_fp4(x, q=None, s=None, scale_layout: str = "rowmajor"):
    """MXFP4 of x bf16 [B?, R, C] in 1x32 blocks along the last axis: q uint8
    [B?, R, C/2] (two codes to a byte, the even column in the low four bits)
    and s uint8 [B?, R, C/32], or [B?, C/128, R, 4] with scale_layout="gemm"
    (an operand of mx_grouped_gemm_mxfp4 as it stands)."""
    import torch
    lib = load_library()
    _require(x, torch.bfloat16, "x")
    B, R, C = _as3d(x)
    lead, dev = (B,) if x.dim() == 3 else (), x.device
    s_shape, layout = _scale_shape(scale_layout, lead, R, C)
    q = _out(q, (*lead, R, C // 2), torch.uint8, dev, "q")
    s = _out(s, s_shape, torch.uint8, dev, "s")
    with _on(dev):
        _check("mx_quantize_rowwise_fp4",
               lib.mx_quantize_rowwise_fp4(_ptr(x), B, R, C, _ptr(q), _ptr(s), layout, _stream(dev)))
    return q, s


def mx_dequantize_fp4(q, s, scale_layout: str = "rowmajor", out=None):
    """The values of MXFP4 codes, bf16 [B?, R, C], from q uint8 [B?, R, C/2]
    and s in either layout.  Exact (a NaN/Inf block's scale byte 255 gives
    NaN)."""
    import torch
    lib = load_library()
    _require(q, torch.uint8, "q")
    _require(s, torch.uint8, "s")
    B, R, C = _as3d(q)
    C *= 2
    lead, dev = (B,) if q.dim() == 3 else (), q.device
    s_shape, layout = _scale_shape(scale_layout, lead, R, C)
    if tuple(s.shape) != s_shape:
        raise ValueError(f"s must have shape {s_shape} for codes {tuple(q.shape)}, got {tuple(s.shape)}")
    _same_device(q, s)
    out = _out(out, (*lead, R, C), torch.bfloat16, dev, "out")
    with _on(dev):
        _check("mx_dequantize_fp4",
               lib.mx_dequantize_fp4(_ptr(q), _ptr(s), B, R, C, layout, _ptr(out), _stream(dev)))
    return out


def mx_quantize_weights_fp4(W, q=None, s=None, q_t=None, s_t=None):
    """MXFP4 of W bf16 [E, N, K] in both orientations from one read:
    (q [E, N, K/2], s [E, K/128, N, 4], q_t [E, K, N/2], s_t [E, N/128, K, 4]),
    blocks along K and along N, scales in the GEMM layout.  N and K must be
    multiples of 128."""
    import torch
    lib = load_library()
    _require(W, torch.bfloat16, "W")
    if W.dim() != 3:
        raise ValueError("W must be [E, N, K]")
    E, N, K = W.shape
    dev = W.device
    q = _out(q, (E, N, K // 2), torch.uint8, dev, "q")
    s = _out(s, (E, K // 128, N, 4), torch.uint8, dev, "s")
    q_t = _out(q_t, (E, K, N // 2), torch.uint8, dev, "q_t")
    s_t = _out(s_t, (E, N // 128, K, 4), torch.uint8, dev, "s_t")
    with _on(dev):
        _check("mx_quantize_weights_fp4", lib.mx_quantize_weights_fp4(_ptr(W), E, N, K, _ptr(q), _ptr(s), _ptr(q_t),
                                                                      _ptr(s_t), _stream(dev)))
    return q, s, q_t, s_t


def _format(fmt, name):
    if fmt not in FORMATS:
        raise ValueError(f"{name} must be 'mxfp8' or 'mxfp4', got {fmt!r}")
    return FORMATS[fmt]


def mx_grouped_gemm_mxfp4(X, sX, Y, sY, offs, x_format: str = "mxfp8", row_map=None, c_rows: Optional[int] = None,
                          out=None, out_dtype=None):
    """C[i,j] = sum_k X[i,k] Y[e][j,k] 2^(sX+sY-254) over the rows i of expert
    e, with MXFP4 weights Y uint8 [E, J, Kc/2] and X uint8 [I, Kc] (x_format
    "mxfp8") or [I, Kc/2] ("mxfp4"); scales in the GEMM layout, sX [Kc/128, I,
    4] and sY [E, Kc/128, J, 4]; offs int32 [E] END offsets of the groups (any
    sizes; rows past the last group are not written).  out bf16, or fp32 with
    out_dtype=torch.float32: [I, J], or with row_map (int32 [I]) [c_rows, J],
    row i stored at row_map[i], as mx_grouped_gemm_mx_rows."""
    import torch
    lib = load_library()
    fmt = _format(x_format, "x_format")
    for t, n in ((X, "X"), (sX, "sX"), (Y, "Y"), (sY, "sY")):
        _require(t, torch.uint8, n)
    _require(offs, torch.int32, "offs")
    if X.dim() != 2 or Y.dim() != 3:
        raise ValueError("X must be [I, Kc] codes and Y [E, J, Kc/2]")
    E, J, Kc = Y.shape[0], Y.shape[1], 2 * Y.shape[2]
    I = X.shape[0]
    if X.shape[1] != (Kc if fmt == 0 else Kc // 2):
        raise ValueError(f"{x_format} rows of X must hold {Kc if fmt == 0 else Kc // 2} bytes for Kc={Kc}, got "
                         f"{X.shape[1]}")
    _offs(offs, E)
    for t, want, n in ((sX, (Kc // 128, I, 4), "sX"), (sY, (E, Kc // 128, J, 4), "sY")):
        if tuple(t.shape) != want:
            raise ValueError(f"{n} must be in the GEMM scale layout {want}, got {tuple(t.shape)}")
    _same_device(X, sX, Y, sY, offs)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    if row_map is None:
        if c_rows is not None:
            raise ValueError("c_rows goes with row_map")
        c_rows = I
    else:
        _require(row_map, torch.int32, "row_map")
        _same_device(X, row_map)
        if tuple(row_map.shape) != (I,):
            raise ValueError(f"row_map must be int32 [{I}] (one entry per row of X), got {tuple(row_map.shape)}")
        if c_rows is None:
            c_rows = out.shape[0] if out is not None else I
    if out is None and row_map is not None:
        out = torch.zeros((c_rows, J), dtype=out_dtype, device=X.device)
    out = _out(out, (c_rows, J), out_dtype, X.device, "out")
    with _on(X.device):
        _check("mx_grouped_gemm_mxfp4",
               lib.mx_grouped_gemm_mxfp4(_ptr(X), _ptr(sX), fmt, _ptr(Y), _ptr(sY), SCALES_GEMM, _ptr(offs), I, J, Kc,
                                         E, _ptr(row_map), int(c_rows), _ptr(out), int(out_dtype == torch.float32),
                                         _stream(X.device)))
    return out


def mx_grouped_mm_fp4_workspace_bytes(M: int, C: int, act_format: str = "mxfp8") -> int:
    return int(load_library().mx_grouped_mm_fp4_workspace_bytes(int(M), int(C), _format(act_format, "act_format")))


def _mm_fp4(name, a, q, s, offs, act_format, out, ws):
    import torch
    lib = load_library()
    fmt = _format(act_format, "act_format")
    _require(a, torch.bfloat16, "A" if name == "mx_grouped_mm_fwd_fp4" else "dOut")
    _require(q, torch.uint8, "weight codes")
    _require(s, torch.uint8, "weight scales")
    if a.dim() != 2 or q.dim() != 3:
        raise ValueError("activations must be [M, C] and weight codes [E, J, C/2]")
    M, C = a.shape
    E, J, C2 = q.shape
    if 2 * C2 != C:
        raise ValueError(f"the activations contract over {C} elements but the weight codes over {2 * C2}")
    _offs(offs, E)
    if C % 128 or tuple(s.shape) != (E, C // 128, J, 4):
        raise ValueError(f"weight scales must be in the GEMM scale layout {(E, C // 128, J, 4)} (contraction a "
                         f"multiple of 128), got {tuple(s.shape)}")
    _same_device(a, q, s, offs)
    out = _out(out, (M, J), torch.bfloat16, a.device, "out")
    need = mx_grouped_mm_fp4_workspace_bytes(M, C, act_format)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=a.device)
    _require(ws, torch.uint8, "ws")
    _same_device(a, ws)
    sizes = (M, J, C) if name == "mx_grouped_mm_fwd_fp4" else (M, C, J)
    with _on(a.device):
        _check(name, getattr(lib, name)(_ptr(a), _ptr(q), _ptr(s), _ptr(offs), *sizes, E, fmt, _ptr(out), _ptr(ws),
                                        ws.numel(), _stream(a.device)))
    return out


def mx_grouped_mm_fwd_fp4(A, qW, sW, offs, act_format: str = "mxfp8", out=None, ws=None):
    """out [M, N] = A [M, K] @ W[e]^T per expert group, W given as (q, s) of
    mx_quantize_weights_fp4 (qW uint8 [E, N, K/2], sW [E, K/128, N, 4]); A bf16
    is quantized to act_format ("mxfp8" or "mxfp4") on the way."""
    return _mm_fp4("mx_grouped_mm_fwd_fp4", A, qW, sW, offs, act_format, out, ws)


def mx_grouped_mm_dgrad_fp4(dOut, qWt, sWt, offs, act_format: str = "mxfp8", out=None, ws=None):
    """dA [M, K] = dOut [M, N] @ W[e] per expert group, W given as (q_t, s_t)
    of mx_quantize_weights_fp4 (qWt uint8 [E, K, N/2], sWt [E, N/128, K, 4])."""
    return _mm_fp4("mx_grouped_mm_dgrad_fp4", dOut, qWt, sWt, offs, act_format, out, ws)


# ---------------------------------------------------------------------------
# A whole MoE layer for a few tokens
# ---------------------------------------------------------------------------
def mx_moe_few_tokens_workspace_bytes(T: int, topk: int, N: int) -> int:
    return int(load_library().mx_moe_few_tokens_workspace_bytes(int(T), int(topk), int(N)))


def mx_moe_few_tokens(x, expert_idx, combine, w13, w2, weight_format: str = "mxfp4", check: bool = True, out=None,
                      ws=None):
    """A gated MoE layer for up to MOE_MAX_TOKENS tokens (decoding):
        out[t] = sum_j combine[t, j] * (silu(g) * u) @ W2[e]^T,
        g, u = x[t] @ W13[e]^T split in halves,  e = expert_idx[t, j].
    x bf16 [T, K]; expert_idx int32 and combine fp32, [T] or [T, k] (k up to
    MOE_MAX_TOPK); w13 = (q, s) of the gate and up weights [E, 2N, K] (gate rows
    first) and w2 = (q, s) of the down weights [E, K, N], the first two results
    of mx_quantize_weights_fp4 (weight_format "mxfp4") or mx_quantize_weights
    ("mxfp8").  K and N multiples of 128.  x and silu(g) * u are quantized to
    MXFP8 in the kernels.  The gate and up sums are fp32, those of the down
    projection as in the grouped products (fp32 with the low bits of small
    products dropped, up to 1.6e-4 of the magnitudes' sum); the weighted sum is
    fp32 and rounded once.  Returns bf16 [T, K].

    check=True reads the routing status (one synchronization) and raises on an
    expert id outside [0, E); with check=False such slots add nothing.  `ws`:
    uint8 scratch of mx_moe_few_tokens_workspace_bytes(T, k, N) bytes, 256-byte
    aligned (allocated when None), not shared by calls that overlap.  With
    check=False, `out` and `ws` given, nothing is allocated or synchronized.
    There is no backward: inputs that require a gradient are refused."""
    import torch
    lib = load_library()
    fmt = _format(weight_format, "weight_format")
    _require(x, torch.bfloat16, "x")
    _require(expert_idx, torch.int32, "expert_idx")
    _require(combine, torch.float32, "combine")
    if torch.is_grad_enabled() and (x.requires_grad or combine.requires_grad):
        raise ValueError("mx_moe_few_tokens has no backward: call it under torch.no_grad(), or train through "
                         "mx_routed_experts")
    (q13, s13), (q2, s2) = w13, w2
    for t, n in ((q13, "w13 codes"), (s13, "w13 scales"), (q2, "w2 codes"), (s2, "w2 scales")):
        _require(t, torch.uint8, n)
    if x.dim() != 2 or q13.dim() != 3:
        raise ValueError("x must be [T, K] and the codes of w13 [E, 2N, K]")
    T, K = x.shape
    if expert_idx.dim() not in (1, 2) or expert_idx.shape[0] != T or expert_idx.shape != combine.shape:
        raise ValueError(f"expert_idx and combine must both be [T={T}] or [T={T}, k], got {tuple(expert_idx.shape)} "
                         f"and {tuple(combine.shape)}")
    topk = 1 if expert_idx.dim() == 1 else expert_idx.shape[1]
    E, N = q13.shape[0], q13.shape[1] // 2
    per = 2 if fmt else 1
    for t, want, n in ((q13, (E, 2 * N, K // per), "w13 codes"), (s13, (E, K // 128, 2 * N, 4), "w13 scales"),
                       (q2, (E, K, N // per), "w2 codes"), (s2, (E, N // 128, K, 4), "w2 scales")):
        if tuple(t.shape) != want:
            raise ValueError(f"{n} must be {want} in {weight_format}, got {tuple(t.shape)}")
    _same_device(x, expert_idx, combine, q13, s13, q2, s2)
    dev = x.device
    out = _out(out, (T, K), torch.bfloat16, dev, "out")
    if ws is None:
        ws = torch.empty(max(mx_moe_few_tokens_workspace_bytes(T, topk, N), 1), dtype=torch.uint8, device=dev)
    else:
        _require(ws, torch.uint8, "ws")
        _same_device(x, ws)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    with _on(dev):
        _check("mx_moe_few_tokens",
               lib.mx_moe_few_tokens(_ptr(x), _ptr(expert_idx), _ptr(combine), _ptr(q13), _ptr(s13), _ptr(q2),
                                     _ptr(s2), fmt, T, topk, K, N, E, _ptr(out), _ptr(status), _ptr(ws), ws.numel(),
                                     _stream(dev)))
    if check and int(status.item()):
        raise ValueError(f"mx_moe_few_tokens: an expert id lies outside [0, {E})")
    return out


# ---------------------------------------------------------------------------
# Around the experts' products: router, activation, weighted sum
# ---------------------------------------------------------------------------
def mx_dequantize(q, s, scale_layout: str = "rowmajor", out=None):
    """The values of MXFP8 codes, bf16 [B?, R, C], from q uint8 [B?, R, C] and s
    in either layout (as mx_dequantize_fp4).  Exact from 2^-126 on; a NaN/Inf
    block's scale byte 255 gives NaN."""
    import torch
    if out is None:
        out = _native().dequantize(q, s, _LAYOUTS.get(scale_layout, -1))
        if out is not None:
            return out
    _require(q, torch.uint8, "q")
    _require(s, torch.uint8, "s")
    B, R, C = _as3d(q)
    lead, dev = (B,) if q.dim() == 3 else (), q.device
    s_shape, layout = _scale_shape(scale_layout, lead, R, C)
    if tuple(s.shape) != s_shape:
        raise ValueError(f"s must have shape {s_shape} for codes {tuple(q.shape)}, got {tuple(s.shape)}")
    _same_device(q, s)
    lib = load_library()
    out = _out(out, tuple(q.shape), torch.bfloat16, dev, "out")
    with _on(dev):
        _check("mx_dequantize", lib.mx_dequantize(_ptr(q), _ptr(s), B, R, C, layout, _ptr(out), _stream(dev)))
    return out


def _type(t, name):
    """MX_BF16 or MX_F32 of a tensor that may be either (contiguous, on the GPU)."""
    import torch
    if isinstance(t, torch.Tensor) and t.dtype == torch.float32:
        _require(t, torch.float32, name)
        return 1
    _require(t, torch.bfloat16, name)
    return 0


def _choice(value, of, name):
    if value not in of:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, of))}, got {value!r}")
    return of[value]


def _router_arguments(logits, k, score, bias, group_score):
    """Checks of the router's operands: codes of the logits' type, the score and the groups' value."""
    import torch
    kind = _type(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if not 0 <= k <= MOE_MAX_TOPK:
        raise ValueError(f"k={k} outside [1, {MOE_MAX_TOPK}]")
    if bias is not None:
        E = logits.shape[1]
        _require(bias, torch.float32, "bias")
        if tuple(bias.shape) != (E,):
            raise ValueError(f"bias must be [{E}] (one per expert), got {tuple(bias.shape)}")
        _same_device(logits, bias)
    return kind, _choice(score, SCORES, "score"), _choice(group_score, GROUP_SCORES, "group_score")


def mx_topk_router_fwd(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
                       group_score: str = "max", renormalize: bool = True, scale: float = 1.0, expert_idx=None,
                       combine=None):
    """(expert_idx int32 [T, k], combine fp32 [T, k]) of the logits (see mx_topk_router), without a gradient."""
    import torch
    lib = load_library()
    kind, sc, gs = _router_arguments(logits, k, score, bias, group_score)
    T, E = logits.shape
    dev = logits.device
    expert_idx = _out(expert_idx, (T, k), torch.int32, dev, "expert_idx")
    combine = _out(combine, (T, k), torch.float32, dev, "combine")
    with _on(dev):
        _check("mx_topk_router_fwd",
               lib.mx_topk_router_fwd(_ptr(logits), kind, _ptr(bias), T, E, k, sc, groups, topk_groups, gs,
                                      int(bool(renormalize)), scale, _ptr(expert_idx), _ptr(combine), _stream(dev)))
    return expert_idx, combine


def mx_topk_router_bwd(logits, expert_idx, combine, dcombine, score: str = "softmax", renormalize: bool = True,
                       scale: float = 1.0, dlogits=None):
    """Gradient of the logits from that of the combine weights (dcombine fp32 [T, k]); expert_idx and combine
    as mx_topk_router_fwd returned them with the same arguments."""
    import torch
    lib = load_library()
    kind = _type(logits, "logits")
    _require(expert_idx, torch.int32, "expert_idx")
    _require(combine, torch.float32, "combine")
    _require(dcombine, torch.float32, "dcombine")
    if logits.dim() != 2 or expert_idx.dim() != 2 or expert_idx.shape[0] != logits.shape[0]:
        raise ValueError("logits must be [T, E] and expert_idx [T, k]")
    if expert_idx.shape != combine.shape or expert_idx.shape != dcombine.shape:
        raise ValueError(f"expert_idx, combine and dcombine must have one shape, got {tuple(expert_idx.shape)}, "
                         f"{tuple(combine.shape)} and {tuple(dcombine.shape)}")
    _same_device(logits, expert_idx, combine, dcombine)
    T, E = logits.shape
    dev = logits.device
    dlogits = _out(dlogits, (T, E), logits.dtype, dev, "dlogits")
    with _on(dev):
        _check("mx_topk_router_bwd",
               lib.mx_topk_router_bwd(_ptr(logits), kind, _ptr(expert_idx), _ptr(combine), _ptr(dcombine), T, E,
                                      expert_idx.shape[1], _choice(score, SCORES, "score"), int(bool(renormalize)),
                                      scale, _ptr(dlogits), _stream(dev)))
    return dlogits


def mx_topk_router(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
                   group_score: str = "max", renormalize: bool = True, scale: float = 1.0):
    """The router: logits fp32 or bf16 [T, E] -> (expert_idx int32 [T, k], combine fp32 [T, k]), what mx_route,
    mx_moe_layer and mx_moe_few_tokens take.  Differentiable in the logits.

        s = softmax(logits) or sigmoid(logits)     score="softmax" / "sigmoid"
        c = s + bias                               bias fp32 [E], for balance: takes part in the choice alone
        expert_idx = the k largest c, largest first, equal ones by index
        combine = scale * s[expert_idx]            divided by their sum with renormalize=True

    groups > 1: the choice is among the experts of the topk_groups best of that many groups of consecutive
    experts; a group counts with its largest c (group_score="max") or the sum of its two largest ("top2").
    The choice is that of 64-bit scores, the weights are fp32.  Experts whose logit is -inf (or the lowest
    finite value of the type) are masked: score 0, chosen after all others; a token with no other expert gets
    weights 0.  E up to 1024, k up to MOE_MAX_TOPK, groups up to ROUTER_MAX_GROUPS, scale in [2^-64, 2^64]."""
    out = _native().topk_router(logits, k, SCORES.get(score, -1), bias, groups, topk_groups,
                                GROUP_SCORES.get(group_score, -1), renormalize, scale)
    if out is not None:
        return out
    from .autograd import mx_topk_router as _f
    return _f(logits, k, score, bias, groups, topk_groups, group_score, renormalize, scale)


def _halves(gu):
    import torch
    _require(gu, torch.bfloat16, "gu")
    if gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError(f"gu must be [M, 2N] (gate columns, then up columns), got {tuple(gu.shape)}")
    return gu.shape[0], gu.shape[1] // 2


def _kept(kept, kept_s, M, N, s_shape):
    import torch
    _require(kept, torch.uint8, "kept")
    _require(kept_s, torch.uint8, "kept_s")
    if tuple(kept.shape) != (M, 2 * N) or tuple(kept_s.shape) != s_shape:
        raise ValueError(f"the checkpoint must be codes {(M, 2 * N)} and scales {s_shape}, got {tuple(kept.shape)} and "
                         f"{tuple(kept_s.shape)}")


def mx_swiglu_fwd(gu, keep: bool = True, h=None, kept=None, kept_s=None):
    """(h bf16 [M, N], kept uint8 [M, 2N], kept_s uint8 [M, 2N/32]) of gu bf16 [M, 2N]: silu(gate) * up and
    the MXFP8 checkpoint of gu that mx_swiglu_bwd reads (None, None with keep=False).  N % 32 == 0."""
    import torch
    lib = load_library()
    M, N = _halves(gu)
    dev = gu.device
    h = _out(h, (M, N), torch.bfloat16, dev, "h")
    if keep:
        kept = _out(kept, (M, 2 * N), torch.uint8, dev, "kept")
        kept_s = _out(kept_s, (M, 2 * N // 32), torch.uint8, dev, "kept_s")
    elif kept is not None or kept_s is not None:
        raise ValueError("kept and kept_s go with keep=True")
    with _on(dev):
        _check("mx_swiglu_fwd", lib.mx_swiglu_fwd(_ptr(gu), M, N, _ptr(h), _ptr(kept), _ptr(kept_s), _stream(dev)))
    return h, kept, kept_s


def mx_swiglu_bwd(dh, kept, kept_s, dgu=None):
    """Gradient of gu, bf16 [M, 2N], from that of h (bf16 [M, N]) at the values of the checkpoint."""
    import torch
    lib = load_library()
    _require(dh, torch.bfloat16, "dh")
    if dh.dim() != 2:
        raise ValueError("dh must be [M, N]")
    M, N = dh.shape
    _kept(kept, kept_s, M, N, (M, 2 * N // 32))
    _same_device(dh, kept, kept_s)
    dev = dh.device
    dgu = _out(dgu, (M, 2 * N), torch.bfloat16, dev, "dgu")
    with _on(dev):
        _check("mx_swiglu_bwd", lib.mx_swiglu_bwd(_ptr(dh), _ptr(kept), _ptr(kept_s), M, N, _ptr(dgu), _stream(dev)))
    return dgu


def mx_swiglu(gu):
    """Differentiable h = silu(gate) * up of gu bf16 [M, 2N] (gate columns first): bf16 [M, N].  N % 32 == 0.

    The backward keeps gu in MXFP8 (2.06 bytes per element of h instead of 4) and is the gradient at the
    values kept: each gate and up value off by at most 1/16 of itself (or, in a block of 32 with a larger
    one, 2^-18 of the largest's power of two; up to 1/8 for values from 7/8 of the next power of two on)."""
    out = _native().swiglu(gu)
    if out is not None:
        return out
    from .autograd import mx_swiglu as _f
    return _f(gu)


def _rows_of(gu, rows, combine, M):
    """Checks of the items that rows stand for; their number."""
    import torch
    if combine is not None:
        _require(combine, torch.float32, "combine")
        _same_device(gu, combine)
    if rows is None:
        if combine is not None and combine.numel() != M:
            raise ValueError(f"without rows combine must hold M={M} weights, got {combine.numel()}")
        return M
    _require(rows, torch.int32, "rows")
    if tuple(rows.shape) != (M,):
        raise ValueError(f"rows must be int32 [{M}] (the item of each row), got {tuple(rows.shape)}")
    _same_device(gu, rows)
    return combine.numel() if combine is not None else (1 << 31) - 1


def mx_swiglu_quantize(gu, rows=None, q=None, s=None):
    """MXFP8 of silu(gate) * up of gu bf16 [M, 2N], (q uint8 [M, N], s uint8 [N/128, M, 4]): X of the next
    grouped product.  rows int32 [M] (of mx_route): rows with a negative entry count as zeros, whatever they
    hold.  N % 128 == 0."""
    import torch
    if q is None and s is None:
        out = _native().swiglu_quantize(gu, rows)
        if out is not None:
            return out
    M, N = _halves(gu)
    n = _rows_of(gu, rows, None, M)
    lib, dev = load_library(), gu.device
    q = _out(q, (M, N), torch.uint8, dev, "q")
    s = _out(s, (N // 128, M, 4), torch.uint8, dev, "s")
    with _on(dev):
        _check("mx_swiglu_quantize",
               lib.mx_swiglu_quantize(_ptr(gu), _ptr(rows), n, M, N, _ptr(q), _ptr(s), _stream(dev)))
    return q, s


def mx_swiglu_quantize_fwd(gu, rows=None, combine=None, ldq: Optional[int] = None, q=None, s=None, q_t=None, s_t=None,
                           kept=None, kept_s=None):
    """The activation between the two products of routed experts, for training: (q, s, q_t, s_t, kept,
    kept_s) of gu bf16 [M, 2N] with the rows of mx_route (None: row r is item r).

      q [M, N], s [N/128, M, 4]         h = silu(gate) * up in 1x32 blocks along N, X of the down product
      q_t [N, ldq], s_t [ldq/128, N, 4] combine[rows[r]] * h in 32x1 blocks along the rows, for the down
                                        weights' gradient (combine fp32, one weight per item; None: 1)
      kept [M, 2N], kept_s [2N/128, M, 4]  the checkpoint of gu in MXFP8, for mx_swiglu_quantize_bwd

    Rows whose entry of `rows` is negative or past the items count as zeros.  M % 32 == 0, N % 128 == 0; ldq
    defaults to M rounded up to 128."""
    import torch
    if q is None and s is None and q_t is None and s_t is None and kept is None and kept_s is None:
        out = _native().swiglu_quantize_fwd(gu, rows, combine, ldq)
        if out is not None:
            return out
    M, N = _halves(gu)
    n = _rows_of(gu, rows, combine, M)
    if ldq is None:
        ldq = (M + 127) // 128 * 128
    lib, dev = load_library(), gu.device
    q = _out(q, (M, N), torch.uint8, dev, "q")
    s = _out(s, (N // 128, M, 4), torch.uint8, dev, "s")
    q_t = _out(q_t, (N, ldq), torch.uint8, dev, "q_t")
    s_t = _out(s_t, (ldq // 128, N, 4), torch.uint8, dev, "s_t")
    kept = _out(kept, (M, 2 * N), torch.uint8, dev, "kept")
    kept_s = _out(kept_s, (2 * N // 128, M, 4), torch.uint8, dev, "kept_s")
    with _on(dev):
        _check("mx_swiglu_quantize_fwd",
               lib.mx_swiglu_quantize_fwd(_ptr(gu), _ptr(rows), _ptr(combine), n, M, N, ldq, _ptr(q), _ptr(s), _ptr(q_t),
                                          _ptr(s_t), _ptr(kept), _ptr(kept_s), _stream(dev)))
    return q, s, q_t, s_t, kept, kept_s


def mx_swiglu_quantize_workspace_bytes(M: int, N: int) -> int:
    return int(load_library().mx_swiglu_quantize_workspace_bytes(int(M), int(N)))


def mx_swiglu_quantize_bwd(dh, kept, kept_s, rows=None, pos=None, combine=None, ldq: Optional[int] = None, q=None, s=None,
                           q_t=None, s_t=None, dcombine=None, ws=None):
    """Its backward: (q [M, 2N], s [2N/128, M, 4], q_t [2N, ldq], s_t [ldq/128, 2N, 4], dcombine) from dh bf16
    [M, N], the gradient of h without the combine weight.  q and q_t are the gradient of gu (combine * dh
    through the activation at the checkpoint's values) in both orientations, dcombine fp32 (the shape of
    combine; None without it) each item's sum over N of dh * h.  rows and pos as mx_route returned them; items
    whose pos is negative get dcombine 0.  `ws`: uint8 scratch of mx_swiglu_quantize_workspace_bytes(M, N)."""
    import torch
    if q is None and s is None and q_t is None and s_t is None and dcombine is None and ws is None:
        out = _native().swiglu_quantize_bwd(dh, kept, kept_s, rows, pos, combine, ldq)
        if out is not None:
            return out
    _require(dh, torch.bfloat16, "dh")
    if dh.dim() != 2:
        raise ValueError("dh must be [M, N]")
    M, N = dh.shape
    _kept(kept, kept_s, M, N, (2 * N // 128, M, 4))
    n = _rows_of(dh, rows, combine, M)
    _same_device(dh, kept, kept_s)
    if combine is None:
        if dcombine is not None:
            raise ValueError("dcombine goes with combine")
        pos = None
    else:
        if (rows is None) != (pos is None):
            raise ValueError("rows and pos go together (both of mx_route)")
        if pos is not None:
            _require(pos, torch.int32, "pos")
            _same_device(dh, pos)
            if pos.numel() != n:
                raise ValueError(f"pos must hold one entry per item ({n}), got {pos.numel()}")
    if ldq is None:
        ldq = (M + 127) // 128 * 128
    lib, dev = load_library(), dh.device
    if combine is not None:
        dcombine = _out(dcombine, tuple(combine.shape), torch.float32, dev, "dcombine")
        if ws is None:
            ws = torch.empty(max(mx_swiglu_quantize_workspace_bytes(M, N), 1), dtype=torch.uint8, device=dev)
        else:
            _require(ws, torch.uint8, "ws")
            _same_device(dh, ws)
    q = _out(q, (M, 2 * N), torch.uint8, dev, "q")
    s = _out(s, (2 * N // 128, M, 4), torch.uint8, dev, "s")
    q_t = _out(q_t, (2 * N, ldq), torch.uint8, dev, "q_t")
    s_t = _out(s_t, (ldq // 128, 2 * N, 4), torch.uint8, dev, "s_t")
    with _on(dev):
        _check("mx_swiglu_quantize_bwd",
               lib.mx_swiglu_quantize_bwd(_ptr(dh), _ptr(kept), _ptr(kept_s), _ptr(rows), _ptr(pos), _ptr(combine), n, M,
                                          N, ldq, _ptr(q), _ptr(s), _ptr(q_t), _ptr(s_t), _ptr(dcombine), _ptr(ws),
                                          0 if ws is None else ws.numel(), _stream(dev)))
    return q, s, q_t, s_t, dcombine


def _combine_sizes(y, combine, pos):
    """Checks of the weighted sum's operands: (type of y, T, k, N)."""
    import torch
    kind = _type(y, "y")
    _require(combine, torch.float32, "combine")
    if y.dim() != 3:
        raise ValueError("y must be [T, k, N] (one row per item)")
    T, k, N = y.shape
    if tuple(combine.shape) != (T, k):
        raise ValueError(f"combine must be [{T}, {k}], got {tuple(combine.shape)}")
    _same_device(y, combine)
    if pos is not None:
        _require(pos, torch.int32, "pos")
        _same_device(y, pos)
        if pos.numel() != T * k:
            raise ValueError(f"pos must hold one entry per item ({T * k}), got {pos.numel()}")
    return kind, T, k, N


def mx_topk_combine_fwd(y, combine, pos=None, out=None):
    """out bf16 [T, N] = sum_j combine[t, j] * y[t, j] (see mx_topk_combine), without a gradient."""
    import torch
    lib = load_library()
    kind, T, k, N = _combine_sizes(y, combine, pos)
    dev = y.device
    out = _out(out, (T, N), torch.bfloat16, dev, "out")
    with _on(dev):
        _check("mx_topk_combine_fwd",
               lib.mx_topk_combine_fwd(_ptr(y), kind, _ptr(combine), _ptr(pos), T, k, N, _ptr(out), _stream(dev)))
    return out


def mx_topk_combine_bwd(dout, y, combine, pos=None, need_dy: bool = True, need_dcombine: bool = True, dy=None,
                        dcombine=None):
    """(dy [T, k, N] in y's type, dcombine fp32 [T, k]) of the weighted sum from dout bf16 [T, N]; None for one
    that is not needed."""
    import torch
    lib = load_library()
    kind, T, k, N = _combine_sizes(y, combine, pos)
    _require(dout, torch.bfloat16, "dout")
    if tuple(dout.shape) != (T, N):
        raise ValueError(f"dout must be [{T}, {N}], got {tuple(dout.shape)}")
    _same_device(y, dout)
    dev = y.device
    dy = _out(dy, (T, k, N), y.dtype, dev, "dy") if need_dy else None
    dcombine = _out(dcombine, (T, k), torch.float32, dev, "dcombine") if need_dcombine else None
    with _on(dev):
        _check("mx_topk_combine_bwd",
               lib.mx_topk_combine_bwd(_ptr(y), kind, _ptr(combine), _ptr(pos), _ptr(dout), T, k, N, _ptr(dy),
                                       _ptr(dcombine), _stream(dev)))
    return dy, dcombine


def mx_topk_combine(y, combine, pos=None):
    """Differentiable weighted sum over a token's experts: out[t] = sum_j combine[t, j] * y[t, j], bf16 [T, N], of
    y bf16 or fp32 [T, k, N] (what mx_routed_experts returns for a top-k router) and combine fp32 [T, k].
    Summed in fp32 in slot order and rounded once.  pos int32 [T * k] (of mx_route): items with a negative
    entry were not routed; their rows are not read, add nothing and get zero gradients.  N % 8 == 0."""
    out = _native().topk_combine(y, combine, pos)
    if out is not None:
        return out
    from .autograd import mx_topk_combine as _f
    return _f(y, combine, pos)


def mx_moe_layer(x, expert_idx, combine, W13, W2, check: bool = True, weights=None, cache=None,
                 weight_format: str = "mxfp8"):
    """A differentiable gated MoE layer on the MXFP8 grouped products (the training form of
    mx_moe_few_tokens):
        out[t] = sum_j combine[t, j] * (silu(g) * u) @ W2[e]^T,
        g, u = x[t] @ W13[e]^T split in halves,  e = expert_idx[t, j]."""
    from .autograd import mx_moe_layer as _f
    return _f(x, expert_idx, combine, W13, W2, check, weights, cache, weight_format)
