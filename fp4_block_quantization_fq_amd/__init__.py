"""Blockwise FP4 (MXFP4 / NVFP4) fake quantization on AMD MI355X (gfx950).

Thin binding over libfq.so (C ABI in include/fq.h): ctypes, and for the row
operators and the feed-forward products, whose calls can be shorter than that
takes, a small extension (csrc/fq_binding.cpp).  Every function here only marshals arguments: shapes, device pointers and the current HIP
stream go to the library, and all arithmetic runs in its HIP kernels.  PyTorch
supplies device memory and streams.  There is no fallback: if libfq.so is
missing or a call fails, an exception is raised.

Tensors: BF16 data is passed as torch.bfloat16 tensors; codes and scales as
torch.uint8; outer scales as torch.float32.  Layouts are those of fq.h.
"""
from __future__ import annotations

import ctypes
import math
import os
from contextlib import nullcontext
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfq.so")

FQ_OK, FQ_ERR_NULL, FQ_ERR_DESC, FQ_ERR_SHAPE, FQ_ERR_ALIGN, FQ_ERR_WORKSPACE, FQ_ERR_DEVICE = range(7)
FQ_SCALE_E8M0, FQ_SCALE_E4M3 = 0, 1
FQ_OUTER_NONE, FQ_OUTER_TENSOR, FQ_OUTER_BLOCK128 = 0, 1, 2
FQ_ROUND_RNE, FQ_ROUND_SR = 0, 1
FQ_AXIS_ROW, FQ_AXIS_COL = 0, 1
FQ_OSCI_BIN_CENTRE, FQ_OSCI_GRID_VALUE = 0, 1
FQ_F8_NONE, FQ_F8_MX, FQ_F8_ROW = 0, 1, 2
FQ_TYPE_BF16, FQ_TYPE_F32 = 0, 1
FQ_STATE_F32, FQ_STATE_F8 = 0, 1
FQ_ACT_NONE, FQ_ACT_RELU, FQ_ACT_SILU, FQ_ACT_GELU = 0, 1, 2, 3
FQ_MOE_MAX_K, FQ_MOE_MAX_ALIGN = 64, 1024
STATE_BLOCK = 128                 # elements under one scale of an 8-bit AdamW state

# every symbol include/fq.h declares
EXPORTED = (
    "fq_desc_mxfp4", "fq_desc_nvfp4", "fq_workspace_size", "fq_quantize",
    "fq_dequantize", "fq_fake_quant", "fq_fake_quant_mask", "fq_ste_backward",
    "fq_ste_backward_mask", "fq_osci_track", "fq_osci_reset", "fq_channel_absmax",
    "fq_select_channels", "fq_fake_quant_retain", "fq_fake_quant_rht",
    "fq_qlinear_workspace_size", "fq_qlinear_fwd", "fq_hadamard",
    "fq_qlinear_bwd_workspace_size", "fq_qlinear_bwd", "fq_status_string",
    "fq_last_error", "fq_version", "fq_fake_quant_noalloc", "fq_qlinear_fwd_retain",
    "fq_qlinear_bwd_retain", "fq_rmsnorm_fwd", "fq_rmsnorm_bwd_workspace_size",
    "fq_rmsnorm_bwd", "fq_moe_rows", "fq_moe_sort_workspace_size", "fq_moe_sort",
    "fq_moe_dispatch", "fq_moe_combine", "fq_moe_combine_bwd", "fq_adamw_step",
    "fq_adamw_plan_size", "fq_adamw_plan", "fq_adamw_step_plan", "fq_f8_encode", "fq_f8_decode",
    "fq_linear_fwd_workspace_size", "fq_linear_fwd", "fq_linear_bwd_workspace_size", "fq_linear_bwd",
    "fq_glu_fwd_workspace_size", "fq_glu_fwd", "fq_glu_bwd_workspace_size", "fq_glu_bwd",
)


class FqDesc(ctypes.Structure):
    _fields_ = [
        ("block_size", ctypes.c_int32),
        ("scale_type", ctypes.c_int32),
        ("outer", ctypes.c_int32),
        ("rounding", ctypes.c_int32),
        ("axis", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("seed", ctypes.c_uint64),
    ]

    def __repr__(self):
        return (f"FqDesc(block_size={self.block_size}, scale_type={self.scale_type}, "
                f"outer={self.outer}, rounding={self.rounding}, axis={self.axis}, "
                f"seed={self.seed})")


class FqAdamWTensor(ctypes.Structure):
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("w_bf16", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("g_type", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("lr_mult", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
    ]


class FqAdamWHyper(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("step", ctypes.c_int64),
        ("seed", ctypes.c_uint64),
        ("grad_scale", ctypes.c_void_p),
        ("state_type", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class FqGate(ctypes.Structure):
    _fields_ = [
        ("act", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("limit", ctypes.c_float),
        ("shift", ctypes.c_float),
    ]


class FqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libfq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m fp4_block_quantization_fq_amd.build` (or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        dp = ctypes.POINTER(FqDesc)
        L.fq_desc_mxfp4.argtypes = []
        L.fq_desc_mxfp4.restype = FqDesc
        L.fq_desc_nvfp4.argtypes = []
        L.fq_desc_nvfp4.restype = FqDesc
        L.fq_workspace_size.argtypes = [dp, i64, i64]
        L.fq_workspace_size.restype = sz
        L.fq_quantize.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, sz, vp]
        L.fq_quantize.restype = ctypes.c_int
        L.fq_dequantize.argtypes = [dp, vp, vp, vp, i64, i64, vp, vp]
        L.fq_dequantize.restype = ctypes.c_int
        L.fq_fake_quant.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]
        L.fq_fake_quant.restype = ctypes.c_int
        L.fq_fake_quant_noalloc.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, vp]
        L.fq_fake_quant_noalloc.restype = ctypes.c_int
        L.fq_ste_backward.argtypes = [dp, vp, vp, vp, vp, i64, i64, vp, vp]
        L.fq_fake_quant_mask.restype = ctypes.c_int
        L.fq_fake_quant_mask.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fq_ste_backward_mask.restype = ctypes.c_int
        f32 = ctypes.c_float
        L.fq_osci_track.argtypes = [vp, vp, vp, vp, vp, vp, i64, ctypes.c_int32, vp]
        L.fq_osci_track.restype = ctypes.c_int
        L.fq_osci_reset.argtypes = [ctypes.POINTER(FqDesc), vp, vp, vp, vp, vp, i64, i64, vp, vp,
                                    vp, vp, f32, ctypes.c_int32, vp]
        L.fq_osci_reset.restype = ctypes.c_int
        L.fq_channel_absmax.argtypes = [vp, i64, i64, vp, vp]
        L.fq_channel_absmax.restype = ctypes.c_int
        L.fq_select_channels.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fq_select_channels.restype = ctypes.c_int
        L.fq_fake_quant_retain.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fq_fake_quant_retain.restype = ctypes.c_int
        L.fq_fake_quant_rht.argtypes = [dp, vp, i64, i64, ctypes.c_int32, ctypes.c_uint64, vp, vp,
                                        vp, vp, vp]
        L.fq_fake_quant_rht.restype = ctypes.c_int
        L.fq_ste_backward_mask.argtypes = [vp, vp, i64, i64, vp, vp]
        L.fq_ste_backward.restype = ctypes.c_int
        L.fq_qlinear_workspace_size.argtypes = [dp, dp, i64, i64, i64]
        L.fq_qlinear_workspace_size.restype = sz
        L.fq_qlinear_fwd.argtypes = [dp, dp, vp, vp, i64, i64, i64, vp, vp, sz, vp]
        L.fq_qlinear_fwd.restype = ctypes.c_int
        i32, u64 = ctypes.c_int32, ctypes.c_uint64
        L.fq_hadamard.argtypes = [vp, i64, i64, i32, i32, u64, vp, vp]
        L.fq_hadamard.restype = ctypes.c_int
        L.fq_qlinear_bwd_workspace_size.argtypes = [dp, dp, dp, i32, i64, i64, i64]
        L.fq_qlinear_bwd_workspace_size.restype = sz
        L.fq_qlinear_bwd.argtypes = [dp, dp, dp, i32, u64, vp, vp, vp, i64, i64, i64, vp, vp, vp,
                                     sz, vp]
        L.fq_qlinear_bwd.restype = ctypes.c_int
        L.fq_qlinear_fwd_retain.argtypes = [dp, dp, vp, vp, i64, i64, i64, vp, vp, vp, vp, sz,
                                            vp]
        L.fq_qlinear_fwd_retain.restype = ctypes.c_int
        L.fq_qlinear_bwd_retain.argtypes = [dp, dp, dp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp,
                                            vp, sz, vp]
        L.fq_qlinear_bwd_retain.restype = ctypes.c_int
        L.fq_rmsnorm_fwd.argtypes = [vp, vp, i32, vp, i32, f32, i64, i64, i32, vp, vp, vp, vp, vp,
                                     vp]
        L.fq_rmsnorm_fwd.restype = ctypes.c_int
        L.fq_rmsnorm_bwd_workspace_size.argtypes = [i64, i64]
        L.fq_rmsnorm_bwd_workspace_size.restype = sz
        L.fq_rmsnorm_bwd.argtypes = [vp, vp, i32, vp, i32, vp, vp, i64, i64, vp, vp, vp, vp, sz,
                                     vp]
        L.fq_rmsnorm_bwd.restype = ctypes.c_int
        L.fq_moe_rows.argtypes = [i64, i64, i64, i64]
        L.fq_moe_rows.restype = i64
        L.fq_moe_sort_workspace_size.argtypes = [i64, i64, i64]
        L.fq_moe_sort_workspace_size.restype = sz
        L.fq_moe_sort.argtypes = [vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, sz, vp]
        L.fq_moe_sort.restype = ctypes.c_int
        L.fq_moe_dispatch.argtypes = [vp, i32, vp, i64, i64, i64, i64, vp, vp, vp, vp]
        L.fq_moe_dispatch.restype = ctypes.c_int
        L.fq_moe_combine.argtypes = [vp, vp, i64, i64, i64, i64, vp, vp, vp]
        L.fq_moe_combine.restype = ctypes.c_int
        L.fq_moe_combine_bwd.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.fq_moe_combine_bwd.restype = ctypes.c_int
        L.fq_adamw_step.argtypes = [ctypes.POINTER(FqAdamWHyper), ctypes.POINTER(FqAdamWTensor),
                                    i64, vp]
        L.fq_adamw_step.restype = ctypes.c_int
        L.fq_adamw_plan_size.argtypes = [i64]
        L.fq_adamw_plan_size.restype = sz
        L.fq_adamw_plan.argtypes = [ctypes.POINTER(FqAdamWTensor), i64, i32, vp, sz]
        L.fq_adamw_plan.restype = ctypes.c_int
        L.fq_adamw_step_plan.argtypes = [ctypes.POINTER(FqAdamWHyper), vp, vp, vp]
        L.fq_adamw_step_plan.restype = ctypes.c_int
        L.fq_f8_encode.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        L.fq_f8_encode.restype = ctypes.c_int
        L.fq_f8_decode.argtypes = [vp, vp, i32, i64, i64, vp, vp]
        L.fq_f8_decode.restype = ctypes.c_int
        gate = ctypes.POINTER(FqGate)
        for op in ("linear", "glu"):
            fn = getattr(L, f"fq_{op}_fwd_workspace_size")
            fn.argtypes, fn.restype = [i64, i64, i64, i64], sz
            fn = getattr(L, f"fq_{op}_bwd_workspace_size")
            fn.argtypes, fn.restype = [i64, i64, i64, i64, i32], sz
        L.fq_linear_fwd.argtypes = [vp, vp, vp, i32, vp, i64, i64, i64, i64, vp, i32, vp, i32, vp, vp,
                                    i32, vp, sz, vp]
        L.fq_linear_fwd.restype = ctypes.c_int
        L.fq_linear_bwd.argtypes = [vp, vp, i32, vp, vp, vp, i32, vp, i64, i64, i64, i64, vp, i32, vp,
                                    vp, i32, vp, vp, sz, vp]
        L.fq_linear_bwd.restype = ctypes.c_int
        L.fq_glu_fwd.argtypes = [gate, vp, vp, vp, i32, i64, i64, i64, i64, vp, vp, i32, vp, vp, vp, sz,
                                 vp]
        L.fq_glu_fwd.restype = ctypes.c_int
        L.fq_glu_bwd.argtypes = [gate, vp, vp, i32, vp, vp, vp, i32, vp, i64, i64, i64, i64, vp, vp, vp,
                                 i32, vp, vp, vp, sz, vp]
        L.fq_glu_bwd.restype = ctypes.c_int
        L.fq_status_string.argtypes = [ctypes.c_int]
        L.fq_status_string.restype = ctypes.c_char_p
        L.fq_last_error.argtypes = []
        L.fq_last_error.restype = ctypes.c_char_p
        L.fq_version.argtypes = []
        L.fq_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int):
    if status != FQ_OK:
        msg = lib().fq_last_error().decode() or lib().fq_status_string(status).decode()
        raise FqError(status, msg)


# ---------------------------------------------------------------------------
# descriptors
# ---------------------------------------------------------------------------

def fq_desc_mxfp4(rounding: int = FQ_ROUND_RNE, axis: int = FQ_AXIS_ROW, seed: int = 0) -> FqDesc:
    d = lib().fq_desc_mxfp4()
    d.rounding, d.axis, d.seed = rounding, axis, seed
    return d


def fq_desc_nvfp4(rounding: int = FQ_ROUND_RNE, axis: int = FQ_AXIS_ROW, seed: int = 0,
                  outer: int = FQ_OUTER_TENSOR) -> FqDesc:
    d = lib().fq_desc_nvfp4()
    d.rounding, d.axis, d.seed, d.outer = rounding, axis, seed, outer
    return d


def block_size(desc: FqDesc) -> int:
    return desc.block_size


# ---------------------------------------------------------------------------
# tensor plumbing
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t, nbytes: int | None = None, name: str = "buffer", elem: int | None = None):
    """Device pointer of a tensor the library will read or write.  The C
    library sees only pointers and sizes, so the binding checks here what it
    cannot: the tensor is on the GPU, contiguous, of the expected element
    size, and holds at least `nbytes` bytes (a smaller buffer would be written
    past its end)."""
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if elem is not None and t.element_size() != elem:
        raise ValueError(f"{name} has {t.element_size()}-byte elements, expected {elem}")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, "
                         f"{nbytes} are needed")
    return ctypes.c_void_p(t.data_ptr())


def _bf16(t, rows: int, cols: int, name: str):
    """A BF16 [rows, cols] operand (2-byte elements)."""
    return _ptr(t, rows * cols * 2, name, elem=2)


def _qptrs(desc, out, rows: int, cols: int):
    """Pointers of the codes, scales and outer outputs, checked against the
    sizes the descriptor implies (each may be None)."""
    if out is None:
        return None, None, None
    s = output_shapes(desc, rows, cols)
    n = lambda shp: 0 if shp is None else math.prod(shp)
    return (_ptr(out.codes, n(s["codes"]), "codes"), _ptr(out.scales, n(s["scales"]), "scales"),
            _ptr(out.outer, 4 * n(s["outer"]), "outer"))


def _stream(stream=None):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _raw_stream(stream) -> int:
    """Handle of a stream, or of the current one of the current device."""
    if stream is not None:
        return stream.cuda_stream
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


_binding_module = None


def _binding():
    """The compiled argument marshalling of the row operators."""
    global _binding_module
    if _binding_module is None:
        lib(), _torch()                    # loaded first: the extension links to them
        from . import _fq_binding
        _binding_module = _fq_binding
    return _binding_module


def _matrix(t, name: str):
    """(rows, cols) of a matrix operand."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape


def _allocating(stream):
    """Outputs and workspaces that a call makes for itself belong to the stream
    it runs on, so their memory is not handed out again while it still works."""
    return nullcontext() if stream is None else _torch().cuda.stream(stream)


@dataclass
class Quantized:
    codes: "object"
    scales: "object"
    outer: "object"


def output_shapes(desc: FqDesc, rows: int, cols: int) -> dict:
    """Shapes of codes, scales and outer for x of shape [rows, cols]."""
    qr, qc = (rows, cols) if desc.axis == FQ_AXIS_ROW else (cols, rows)
    B = desc.block_size
    shapes = {"codes": (qr, qc // 2), "scales": (qr, qc // B)}
    if desc.outer == FQ_OUTER_TENSOR:
        shapes["outer"] = (1,)
    elif desc.outer == FQ_OUTER_BLOCK128:
        shapes["outer"] = (qr, qc // 128)
    else:
        shapes["outer"] = None
    return shapes


def alloc_outputs(desc: FqDesc, rows: int, cols: int, device) -> Quantized:
    torch = _torch()
    s = output_shapes(desc, rows, cols)
    codes = torch.empty(s["codes"], dtype=torch.uint8, device=device)
    scales = torch.empty(s["scales"], dtype=torch.uint8, device=device)
    outer = None if s["outer"] is None else torch.empty(s["outer"], dtype=torch.float32, device=device)
    return Quantized(codes, scales, outer)


def workspace(desc: FqDesc, rows: int, cols: int, device):
    torch = _torch()
    n = lib().fq_workspace_size(ctypes.byref(desc), rows, cols)
    return torch.empty((max(n, 16),), dtype=torch.uint8, device=device), n


# ---------------------------------------------------------------------------
# the five operations
# ---------------------------------------------------------------------------

def fq_quantize(desc: FqDesc, x, out: Quantized | None = None, ws=None, stream=None) -> Quantized:
    rows, cols = x.shape
    if out is None:
        out = alloc_outputs(desc, rows, cols, x.device)
    if ws is None:
        ws, nbytes = workspace(desc, rows, cols, x.device)
    else:
        nbytes = ws.numel() * ws.element_size()
    codes, scales, outer = _qptrs(desc, out, rows, cols)
    _check(lib().fq_quantize(ctypes.byref(desc), _bf16(x, rows, cols, "x"), rows, cols, codes,
                             scales, outer, _ptr(ws, nbytes, "ws"), nbytes, _stream(stream)))
    return out


def fq_dequantize(desc: FqDesc, q: Quantized, rows: int, cols: int, y=None, stream=None):
    torch = _torch()
    if y is None:
        y = torch.empty((rows, cols), dtype=torch.bfloat16, device=q.codes.device)
    codes, scales, outer = _qptrs(desc, q, rows, cols)
    _check(lib().fq_dequantize(ctypes.byref(desc), codes, scales, outer, rows, cols,
                               _bf16(y, rows, cols, "y"), _stream(stream)))
    return y


def fq_fake_quant(desc: FqDesc, x, y=None, out: Quantized | None = None, ws=None,
                  stream=None):
    """y = dequantize(quantize(x)); also fills `out` (codes, scales, outer) if
    given.  Returns y."""
    torch = _torch()
    rows, cols = x.shape
    if y is None:
        y = torch.empty_like(x)
    if ws is None:
        ws, nbytes = workspace(desc, rows, cols, x.device)
    else:
        nbytes = ws.numel() * ws.element_size()
    codes, scales, outer = _qptrs(desc, out, rows, cols)
    _check(lib().fq_fake_quant(ctypes.byref(desc), _bf16(x, rows, cols, "x"), rows, cols,
                               _bf16(y, rows, cols, "y"), codes, scales, outer,
                               _ptr(ws, nbytes, "ws"), nbytes, _stream(stream)))
    return y


def fq_fake_quant_noalloc(desc: FqDesc, x, y, out: Quantized | None = None, stream=None):
    """fq_fake_quant with the library's own per-GPU scratch instead of a
    workspace (the C call allocates nothing; y and out are the caller's).
    Returns y."""
    rows, cols = x.shape
    codes, scales, outer = _qptrs(desc, out, rows, cols)
    _check(lib().fq_fake_quant_noalloc(ctypes.byref(desc), _bf16(x, rows, cols, "x"), rows, cols,
                                       _bf16(y, rows, cols, "y"), codes, scales, outer,
                                       _stream(stream)))
    return y


def fq_fake_quant_mask(desc: FqDesc, x, y=None, out: Quantized | None = None, keep=None,
                       ws=None, stream=None):
    """fq_fake_quant that also writes the STE keep mask (uint8 [rows, cols/8],
    layout of x, bit c mod 8 of byte (r, c/8) set where element (r, c) was
    kept).  Returns (y, keep)."""
    torch = _torch()
    rows, cols = x.shape
    if y is None:
        y = torch.empty_like(x)
    if keep is None:
        keep = torch.empty((rows, cols // 8), dtype=torch.uint8, device=x.device)
    if ws is None:
        ws, nbytes = workspace(desc, rows, cols, x.device)
    else:
        nbytes = ws.numel() * ws.element_size()
    codes, scales, outer = _qptrs(desc, out, rows, cols)
    _check(lib().fq_fake_quant_mask(ctypes.byref(desc), _bf16(x, rows, cols, "x"), rows, cols,
                                    _bf16(y, rows, cols, "y"), codes, scales, outer,
                                    _ptr(keep, rows * cols // 8, "keep"),
                                    _ptr(ws, nbytes, "ws"), nbytes, _stream(stream)))
    return y, keep


def fq_ste_backward_mask(keep, dy, dx=None, stream=None):
    """dx = dy where the keep bit is set, else +0.  Returns dx."""
    torch = _torch()
    rows, cols = dy.shape
    if dx is None:
        dx = torch.empty_like(dy)
    _check(lib().fq_ste_backward_mask(_ptr(keep, rows * cols // 8, "keep"),
                                      _bf16(dy, rows, cols, "dy"), rows, cols,
                                      _bf16(dx, rows, cols, "dx"), _stream(stream)))
    return dx


def osci_state(n: int, device):
    """OsciReset state for n weights: w_prev, dist_m, dist_q FP32 and q_prev BF16."""
    torch = _torch()
    return {"w_prev": torch.zeros(n, dtype=torch.float32, device=device),
            "q_prev": torch.zeros(n, dtype=torch.bfloat16, device=device),
            "dist_m": torch.zeros(n, dtype=torch.float32, device=device),
            "dist_q": torch.zeros(n, dtype=torch.float32, device=device)}


def _osci_ptrs(w, q, st: dict, n: int):
    return (_ptr(w, 4 * n, "w", elem=4), _ptr(q, 2 * n, "q", elem=2),
            _ptr(st["w_prev"], 4 * n, "w_prev", elem=4), _ptr(st["q_prev"], 2 * n, "q_prev", elem=2),
            _ptr(st["dist_m"], 4 * n, "dist_m", elem=4), _ptr(st["dist_q"], 4 * n, "dist_q", elem=4))


def fq_osci_track(w, q, st: dict, first: bool = False, stream=None):
    """One step of the oscillation tracker (w FP32 master, q BF16 quantized)."""
    n = w.numel()
    _check(lib().fq_osci_track(*_osci_ptrs(w, q, st, n), n, 1 if first else 0, _stream(stream)))


def fq_osci_reset(w, q, st: dict, tau: float, desc=None, quant=None,
                  target: int = FQ_OSCI_BIN_CENTRE, stream=None):
    """The OsciReset check: oscillating master weights (in place in w, an FP32
    [rows, cols] tensor) go to the centre of their current quantization bin,
    read from `quant` (the Quantized outputs of the quantization with `desc`
    that gave q), or with target=FQ_OSCI_GRID_VALUE to q itself; every
    element starts a new window."""
    assert w.dim() == 2, "w must be [rows, cols]"
    rows, cols = w.shape
    n = rows * cols
    ptrs = _osci_ptrs(w, q, st, n)
    if target == FQ_OSCI_GRID_VALUE:
        d, codes, scales, outer = None, None, None, None
    else:
        d = ctypes.byref(desc)
        codes, scales, outer = _qptrs(desc, quant, rows, cols)
    _check(lib().fq_osci_reset(d, ptrs[0], ptrs[1], codes, scales, outer, rows, cols, *ptrs[2:],
                               ctypes.c_float(tau), target, _stream(stream)))


def fq_channel_absmax(x, amax=None, stream=None):
    """Fold max |x[:, c]| (BF16 magnitude bits) into amax [cols] (int32
    tensor, zeros if not given).  Returns amax."""
    torch = _torch()
    rows, cols = x.shape
    if amax is None:
        amax = torch.zeros(cols, dtype=torch.int32, device=x.device)
    _check(lib().fq_channel_absmax(_bf16(x, rows, cols, "x"), rows, cols,
                                   _ptr(amax, 4 * cols, "amax", elem=4), _stream(stream)))
    return amax


def fq_select_channels(amax, k: int, stream=None):
    """The k largest channels: (retain uint8 [cols/8] bit mask, chan_scale
    float32 [cols])."""
    torch = _torch()
    cols = amax.numel()
    retain = torch.empty(cols // 8, dtype=torch.uint8, device=amax.device)
    scale = torch.empty(cols, dtype=torch.float32, device=amax.device)
    _check(lib().fq_select_channels(_ptr(amax, 4 * cols, "amax", elem=4), cols, k,
                                    _ptr(retain), _ptr(scale), _stream(stream)))
    return retain, scale


def fq_fake_quant_retain(desc: FqDesc, x, retain, chan_scale, y=None,
                         out: Quantized | None = None, ws=None, stream=None):
    """Fake quantization (either axis, any format) with the retained channels
    (columns of x) in FP8.  Returns y."""
    torch = _torch()
    rows, cols = x.shape
    if y is None:
        y = torch.empty_like(x)
    if ws is None:
        ws, nbytes = workspace(desc, rows, cols, x.device)
    else:
        nbytes = ws.numel() * ws.element_size()
    codes, scales, outer = _qptrs(desc, out, rows, cols)
    _check(lib().fq_fake_quant_retain(ctypes.byref(desc), _bf16(x, rows, cols, "x"), rows, cols,
                                      _bf16(y, rows, cols, "y"), codes, scales, outer,
                                      _ptr(retain, cols // 8, "retain"),
                                      _ptr(chan_scale, 4 * cols, "chan_scale", elem=4),
                                      _ptr(ws, nbytes, "ws"), nbytes, _stream(stream)))
    return y


def fq_fake_quant_rht(desc: FqDesc, x, rht_block: int, rht_seed: int, y=None,
                      out: Quantized | None = None, stream=None):
    """Fake quantization of the random Hadamard rotation of x along the
    quantization axis, in one pass.  Returns y."""
    torch = _torch()
    rows, cols = x.shape
    if y is None:
        y = torch.empty_like(x)
    codes, scales, outer = _qptrs(desc, out, rows, cols)
    _check(lib().fq_fake_quant_rht(ctypes.byref(desc), _bf16(x, rows, cols, "x"), rows, cols,
                                   rht_block, rht_seed, _bf16(y, rows, cols, "y"), codes, scales,
                                   outer, _stream(stream)))
    return y


def fq_ste_backward(desc: FqDesc, x, q: Quantized, dy, dx=None, stream=None):
    torch = _torch()
    rows, cols = x.shape
    if dx is None:
        dx = torch.empty_like(dy)
    _, scales, outer = _qptrs(desc, Quantized(None, q.scales, q.outer), rows, cols)
    _check(lib().fq_ste_backward(ctypes.byref(desc), _bf16(x, rows, cols, "x"), scales, outer,
                                 _bf16(dy, rows, cols, "dy"), rows, cols,
                                 _bf16(dx, rows, cols, "dx"), _stream(stream)))
    return dx


def qlinear_workspace(desc_x: FqDesc, desc_w: FqDesc, M: int, K: int, N: int, device):
    torch = _torch()
    n = lib().fq_qlinear_workspace_size(ctypes.byref(desc_x), ctypes.byref(desc_w), M, K, N)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def qlinear_workspace_views(ws, M: int, K: int, N: int):
    """(X_hat [M, K], W_hat^T [N, K]) views into a qlinear workspace."""
    torch = _torch()
    off = (M * K * 2 + 255) // 256 * 256
    xhat = ws[: M * K * 2].view(torch.bfloat16).view(M, K)
    what_t = ws[off: off + N * K * 2].view(torch.bfloat16).view(N, K)
    return xhat, what_t


def qlinear_workspace_mx_views(ws, M: int, K: int, N: int):
    """(X codes [M, K/2], X scales [M, K/32], W^T codes [N, K/2], W^T scales
    [N, K/32]) in a qlinear workspace used by an MXFP4 x MXFP4 linear."""
    r = lambda v: (v + 255) // 256 * 256
    c1 = r(M * K // 2)
    c2 = c1 + r(M * K // 32)
    c3 = c2 + r(N * K // 2)
    return (ws[: M * K // 2].view(M, K // 2), ws[c1: c1 + M * K // 32].view(M, K // 32),
            ws[c2: c2 + N * K // 2].view(N, K // 2), ws[c3: c3 + N * K // 32].view(N, K // 32))


def fq_qlinear_fwd(desc_x: FqDesc, desc_w: FqDesc, x, w, y=None, ws=None, stream=None):
    """Y [M, N] = FQ(X) @ FQ(W) (BF16 out, FP32 accumulation)."""
    torch = _torch()
    M, K = x.shape
    K2, N = w.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {x.shape} @ {w.shape}")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = qlinear_workspace(desc_x, desc_w, M, K, N, x.device)
    _check(lib().fq_qlinear_fwd(ctypes.byref(desc_x), ctypes.byref(desc_w), _bf16(x, M, K, "x"),
                                _bf16(w, K, N, "w"), M, K, N, _bf16(y, M, N, "y"),
                                _ptr(ws, None, "ws", elem=1), ws.numel(), _stream(stream)))
    return y


def fq_hadamard(x, block: int, axis: int = FQ_AXIS_ROW, seed: int = 0, y=None, stream=None):
    """Random Hadamard transform of a [R, C] BF16 tensor in blocks of 16 or 128."""
    torch = _torch()
    rows, cols = x.shape
    if y is None:
        y = torch.empty_like(x)
    _check(lib().fq_hadamard(_bf16(x, rows, cols, "x"), rows, cols, axis, block, seed,
                             _bf16(y, rows, cols, "y"), _stream(stream)))
    return y


def qlinear_bwd_workspace(desc_x: FqDesc, desc_w: FqDesc, desc_g: FqDesc, M: int, K: int,
                          N: int, device, rht_block: int = 0):
    torch = _torch()
    n = lib().fq_qlinear_bwd_workspace_size(ctypes.byref(desc_x), ctypes.byref(desc_w),
                                            ctypes.byref(desc_g), rht_block, M, K, N)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def fq_qlinear_bwd(desc_x: FqDesc, desc_w: FqDesc, desc_g: FqDesc, x, w, dy, dx=None, dw=None,
                   ws=None, stream=None, rht_block: int = 0, rht_seed: int = 0):
    """(dX [M, K], dW [K, N]) of Y = FQ(X) @ FQ(W) for the upstream gradient dY [M, N];
    rht_block 16/128 rotates each product's operands by the random Hadamard transform."""
    torch = _torch()
    M, K = x.shape
    K2, N = w.shape
    if K2 != K or tuple(dy.shape) != (M, N):
        raise ValueError(f"shapes differ: x {tuple(x.shape)}, w {tuple(w.shape)}, dy {tuple(dy.shape)}")
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
    if dw is None:
        dw = torch.empty((K, N), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = qlinear_bwd_workspace(desc_x, desc_w, desc_g, M, K, N, x.device, rht_block)
    _check(lib().fq_qlinear_bwd(ctypes.byref(desc_x), ctypes.byref(desc_w), ctypes.byref(desc_g),
                                rht_block, rht_seed, _bf16(x, M, K, "x"), _bf16(w, K, N, "w"),
                                _bf16(dy, M, N, "dy"), M, K, N, _bf16(dx, M, K, "dx"),
                                _bf16(dw, K, N, "dw"), _ptr(ws, None, "ws", elem=1), ws.numel(),
                                _stream(stream)))
    return dx, dw


def fq_qlinear_fwd_retain(desc_x: FqDesc, desc_w: FqDesc, x, w, retain, chan_scale, y=None,
                          ws=None, stream=None):
    """Y = FQ(X) @ FQ(W) with X's retained channels (retain [K/8], chan_scale
    [K]) in FP8."""
    torch = _torch()
    M, K = x.shape
    K2, N = w.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {x.shape} @ {w.shape}")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = qlinear_workspace(desc_x, desc_w, M, K, N, x.device)
    _check(lib().fq_qlinear_fwd_retain(ctypes.byref(desc_x), ctypes.byref(desc_w),
                                       _bf16(x, M, K, "x"), _bf16(w, K, N, "w"), M, K, N,
                                       _ptr(retain, K // 8, "retain"),
                                       _ptr(chan_scale, 4 * K, "chan_scale", elem=4),
                                       _bf16(y, M, N, "y"), _ptr(ws, None, "ws", elem=1),
                                       ws.numel(), _stream(stream)))
    return y


def fq_qlinear_bwd_retain(desc_x: FqDesc, desc_w: FqDesc, desc_g: FqDesc, x, w, dy, retain,
                          chan_scale, dx=None, dw=None, ws=None, stream=None):
    """(dX, dW) of the linear with X's retained channels in FP8 in the forward
    and the backward."""
    torch = _torch()
    M, K = x.shape
    K2, N = w.shape
    if K2 != K or tuple(dy.shape) != (M, N):
        raise ValueError(f"shapes differ: x {tuple(x.shape)}, w {tuple(w.shape)}, dy {tuple(dy.shape)}")
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
    if dw is None:
        dw = torch.empty((K, N), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = qlinear_bwd_workspace(desc_x, desc_w, desc_g, M, K, N, x.device, 0)
    _check(lib().fq_qlinear_bwd_retain(ctypes.byref(desc_x), ctypes.byref(desc_w),
                                       ctypes.byref(desc_g), _bf16(x, M, K, "x"),
                                       _bf16(w, K, N, "w"), _bf16(dy, M, N, "dy"), M, K, N,
                                       _ptr(retain, K // 8, "retain"),
                                       _ptr(chan_scale, 4 * K, "chan_scale", elem=4),
                                       _bf16(dx, M, K, "dx"), _bf16(dw, K, N, "dw"),
                                       _ptr(ws, None, "ws", elem=1), ws.numel(), _stream(stream)))
    return dx, dw


# ---------------------------------------------------------------------------
# around the linears: norm, expert sorting, optimizer
# ---------------------------------------------------------------------------

def _type_of(t, name: str) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return FQ_TYPE_BF16
    if t.dtype == torch.float32:
        return FQ_TYPE_F32
    raise ValueError(f"{name} must be bfloat16 or float32, not {t.dtype}")


def _typed(t, dtype, n: int, name: str):
    """Pointer of an optional operand of exactly this dtype, `n` elements at least."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    return _ptr(t, n * t.element_size(), name)


def fq_rmsnorm_fwd(x, gamma, eps: float, res=None, f8: int = FQ_F8_NONE, h=None, y=None,
                   codes=None, scales=None, rstd=None, stream=None):
    """Residual addition and root-mean-square norm of x BF16 [rows, cols].

    With a residual `res` (BF16 or FP32, the stream) h = x + res in its type;
    h may be res itself.  f8=FQ_F8_NONE writes y (BF16); otherwise codes (E4M3,
    uint8) and scales, and y only if given (the values they stand for).  rstd
    (FP32 [rows], for the backward) is written if given.  Returns (h, y) without
    f8 and (h, codes, scales) with it; h is None without a residual."""
    if res is not None and h is None or (y is None if f8 == FQ_F8_NONE
                                         else codes is None or scales is None):
        torch = _torch()
        rows, cols = _matrix(x, "x")
        with _allocating(stream):
            if res is not None and h is None:
                h = torch.empty_like(res)
            if f8 == FQ_F8_NONE:
                y = torch.empty_like(x) if y is None else y
            else:
                if codes is None:
                    codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
                if scales is None:
                    scales = (torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
                              if f8 == FQ_F8_MX else
                              torch.empty(rows, dtype=torch.float32, device=x.device))
    st = (_binding_module or _binding()).rmsnorm_fwd(x, gamma, eps, res, f8, h, y, codes, scales,
                                                     rstd, stream)
    if st:
        _check(st)
    return (h, y) if f8 == FQ_F8_NONE else (h, codes, scales)


def rmsnorm_bwd_workspace(rows: int, cols: int, device):
    torch = _torch()
    n = lib().fq_rmsnorm_bwd_workspace_size(rows, cols)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def fq_rmsnorm_bwd(dy, h, gamma, rstd, dres=None, dh=None, dx=None, dgamma=None, ws=None,
                   need_dgamma: bool = True, stream=None):
    """(dh, dgamma) of the norm of h (the forward's h, or its x without a
    residual) for the gradient dy of its output; dres is added to dh (and may
    be dh).  dx, if given, receives dh in BF16 beside an FP32 stream.
    need_dgamma=False leaves dgamma out (None)."""
    if not need_dgamma:
        dgamma = ws = None
    if dh is None or (need_dgamma and (dgamma is None or ws is None)):
        torch = _torch()
        rows, cols = _matrix(dy, "dy")
        with _allocating(stream):
            if dh is None:
                dh = torch.empty_like(h)
            if need_dgamma and dgamma is None:
                dgamma = torch.empty(cols, dtype=torch.float32, device=dy.device)
            if need_dgamma and ws is None:
                ws = rmsnorm_bwd_workspace(rows, cols, dy.device)
    st = (_binding_module or _binding()).rmsnorm_bwd(dy, h, gamma, rstd, dres, dh, dx, dgamma, ws,
                                                     stream)
    if st:
        _check(st)
    return dh, dgamma


@dataclass
class MoeSorted:
    """Where the assignments are in the sorted order: int32 offsets [experts + 1],
    pos [tokens, k] and src [rows]."""
    offsets: "object"
    pos: "object"
    src: "object"


def moe_rows(tokens: int, k: int, experts: int, align: int = 1) -> int:
    """Rows of the sorted order's buffers (what its segments take at most)."""
    n = lib().fq_moe_rows(tokens, k, experts, align)
    if n == 0:
        _check(FQ_ERR_SHAPE)
    return n


def moe_sort_workspace(tokens: int, k: int, experts: int, device):
    torch = _torch()
    n = lib().fq_moe_sort_workspace_size(tokens, k, experts)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def fq_moe_sort(experts_of, experts: int, align: int = 1, out: MoeSorted | None = None, ws=None,
                stream=None) -> MoeSorted:
    """Sort the assignments experts_of (int32 [tokens, k]) by expert, each
    expert's segment padded to a multiple of `align` rows."""
    if out is None or ws is None:
        torch = _torch()
        tokens, k = _matrix(experts_of, "experts_of")
        dev = experts_of.device
        with _allocating(stream):
            if out is None:
                out = MoeSorted(
                    torch.empty(experts + 1, dtype=torch.int32, device=dev),
                    torch.empty((tokens, k), dtype=torch.int32, device=dev),
                    torch.empty(moe_rows(tokens, k, experts, align), dtype=torch.int32,
                                device=dev))
            if ws is None:
                ws = moe_sort_workspace(tokens, k, experts, dev)
    st = (_binding_module or _binding()).moe_sort(experts_of, experts, align, out.offsets, out.pos,
                                                  out.src, ws, stream)
    if st:
        _check(st)
    return out


def fq_moe_dispatch(x, q: MoeSorted, f8: int = FQ_F8_NONE, scales=None, y=None, stream=None):
    """Rows of the tokens in the sorted order (BF16 [rows, cols], 0 in padding):
    x BF16 [tokens, cols], or the codes of 8-bit rows with their scales."""
    if y is None:
        with _allocating(stream):
            y = _torch().empty((q.src.numel(), _matrix(x, "x")[1]), dtype=_torch().bfloat16,
                               device=x.device)
    st = (_binding_module or _binding()).moe_dispatch(x, f8, scales, q.pos, q.src, y, stream)
    if st:
        _check(st)
    return y


def fq_moe_combine(y, q: MoeSorted, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * y[row of (t, j)] (weights None: ones, the
    backward of fq_moe_dispatch)."""
    if out is None:
        with _allocating(stream):
            out = _torch().empty((_matrix(q.pos, "pos")[0], _matrix(y, "y")[1]), dtype=_torch().bfloat16,
                                 device=y.device)
    st = (_binding_module or _binding()).moe_combine(y, weights, q.pos, q.src, out, stream)
    if st:
        _check(st)
    return out


def fq_moe_combine_bwd(dout, y, q: MoeSorted, weights, dy=None, dweights=None, stream=None):
    """(dy [rows, cols] BF16, dweights [tokens, k] FP32) of fq_moe_combine."""
    if dy is None or dweights is None:
        torch = _torch()
        with _allocating(stream):
            if dy is None:
                dy = torch.empty((q.src.numel(), _matrix(dout, "dout")[1]), dtype=torch.bfloat16,
                                 device=dout.device)
            if dweights is None:
                dweights = torch.empty(tuple(q.pos.shape), dtype=torch.float32,
                                       device=dout.device)
    st = (_binding_module or _binding()).moe_combine_bwd(dout, y, weights, q.pos, q.src, dy,
                                                         dweights, stream)
    if st:
        _check(st)
    return dy, dweights


@dataclass
class AdamWTensor:
    """One tensor of an AdamW step: FP32 master w, gradient g (BF16 or FP32),
    moments m and v (FP32, or uint8 codes with m_scale and v_scale), and the
    BF16 copy of w that the linears read (may be None)."""
    w: "object"
    g: "object"
    m: "object"
    v: "object"
    w_bf16: "object" = None
    m_scale: "object" = None
    v_scale: "object" = None
    weight_decay: float = 0.0
    lr_mult: float = 1.0


def adamw_state(n: int, device, f8: bool = False) -> dict:
    """Moments of n elements before the first step (keywords of AdamWTensor)."""
    torch = _torch()
    dtype = torch.uint8 if f8 else torch.float32
    st = {k: torch.zeros(n, dtype=dtype, device=device) for k in ("m", "v")}
    if f8:
        for k in ("m_scale", "v_scale"):
            st[k] = torch.zeros(-(-n // STATE_BLOCK), dtype=torch.float32, device=device)
    return st


class AdamWPlan:
    """The tensors of an optimizer as the library takes them, checked once and
    laid out in device memory, so that a step is one launch.  It holds the
    tensors it was made from; their contents may change between steps, the
    tensors may not.  Making one copies its table, so not while a graph is
    captured; a captured step reads the table at every replay: keep the plan as
    long as the graph."""

    def __init__(self, tensors):
        torch = _torch()
        self.tensors = list(tensors)
        array = (FqAdamWTensor * len(self.tensors))()
        self.f8 = bool(self.tensors) and self.tensors[0].m.dtype != torch.float32
        for i, (s, t) in enumerate(zip(array, self.tensors)):
            n, name = t.w.numel(), f"tensor {i}: "
            s.n = n
            s.w = _typed(t.w, torch.float32, n, name + "w")
            s.w_bf16 = _typed(t.w_bf16, torch.bfloat16, n, name + "w_bf16")
            s.g = _ptr(t.g, n * t.g.element_size(), name + "g")
            s.g_type = _type_of(t.g, name + "g")
            if self.f8:
                blocks = -(-n // STATE_BLOCK)
                s.m, s.v = _ptr(t.m, n, name + "m", elem=1), _ptr(t.v, n, name + "v", elem=1)
                s.m_scale = _typed(t.m_scale, torch.float32, blocks, name + "m_scale")
                s.v_scale = _typed(t.v_scale, torch.float32, blocks, name + "v_scale")
            else:
                s.m = _typed(t.m, torch.float32, n, name + "m")
                s.v = _typed(t.v, torch.float32, n, name + "v")
            s.lr_mult, s.weight_decay = t.lr_mult, t.weight_decay
        self.state_type = FQ_STATE_F8 if self.f8 else FQ_STATE_F32
        nbytes = lib().fq_adamw_plan_size(len(array))
        self.host = torch.empty(nbytes, dtype=torch.uint8, device="cpu")        # 64-byte aligned
        self.address = self.host.data_ptr()
        _check(lib().fq_adamw_plan(array, len(array), self.state_type, self.address, nbytes))
        self.device = self.host.to(self.tensors[0].w.device) if self.tensors else None
        self.stream = _raw_stream(None) if self.tensors else 0      # whose memory the table is
        self._others = set()

    def _read_on(self, stream):
        """The table's memory belongs to the stream that it was made on; a step on
        another one makes it that one's too, so that it is not handed out again
        while that step still takes its pointers from it."""
        raw = _raw_stream(stream)
        if self.device is not None and raw not in self._others:
            self.device.record_stream(_torch().cuda.current_stream() if stream is None else stream)
            self._others.add(raw)


def adamw_plan(tensors) -> AdamWPlan:
    return AdamWPlan(tensors)


def fq_adamw_step(plan: AdamWPlan, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
                  eps: float = 1e-8, grad_scale=None, seed: int = 0, stream=None):
    """One AdamW step (in place) over a plan's tensors.  step counts from 1;
    grad_scale is an FP32 device scalar the gradients are multiplied by; seed
    keys the stochastic rounding of 8-bit moments."""
    st = (_binding_module or _binding()).adamw_step(
        plan.address, plan.device, plan.state_type, lr, beta1, beta2, eps, step, seed, grad_scale,
        stream, plan.stream, plan._read_on)
    if st:
        _check(st)


# ---------------------------------------------------------------------------
# the feed-forward products, and checkpoints in 8 bits
# ---------------------------------------------------------------------------

def _f8_scales(rows: int, cols: int, f8: int, device):
    torch = _torch()
    if f8 == FQ_F8_MX:
        return torch.empty((rows, cols // 32), dtype=torch.uint8, device=device)
    return torch.empty(rows, dtype=torch.float32, device=device)


def fq_f8_encode(x, f8: int, codes=None, scales=None, stream=None):
    """x BF16 [rows, cols] as 8-bit rows: (codes uint8 [rows, cols], scales)."""
    if codes is None or scales is None:
        rows, cols = _matrix(x, "x")
        with _allocating(stream):
            if codes is None:
                codes = _torch().empty((rows, cols), dtype=_torch().uint8, device=x.device)
            if scales is None:
                scales = _f8_scales(rows, cols, f8, x.device)
    st = (_binding_module or _binding()).f8_encode(x, f8, codes, scales, stream)
    if st:
        _check(st)
    return codes, scales


def fq_f8_decode(codes, scales, f8: int, y=None, stream=None):
    """The values that 8-bit rows stand for, in BF16."""
    if y is None:
        with _allocating(stream):
            y = _torch().empty(_matrix(codes, "codes"), dtype=_torch().bfloat16, device=codes.device)
    st = (_binding_module or _binding()).f8_decode(codes, scales, f8, y, stream)
    if st:
        _check(st)
    return y


def _product_workspace(size: int, device):
    return _torch().empty((size,), dtype=_torch().uint8, device=device)


def linear_fwd_workspace(rows: int, k: int, n: int, experts: int, device):
    return _product_workspace(lib().fq_linear_fwd_workspace_size(rows, k, n, experts), device)


def glu_fwd_workspace(rows: int, k: int, n: int, experts: int, device):
    return _product_workspace(lib().fq_glu_fwd_workspace_size(rows, k, n, experts), device)


def linear_bwd_workspace(rows: int, k: int, n: int, experts: int, device, x_f8: int = FQ_F8_NONE):
    return _product_workspace(lib().fq_linear_bwd_workspace_size(rows, k, n, experts, x_f8), device)


def glu_bwd_workspace(rows: int, k: int, n: int, experts: int, device, x_f8: int = FQ_F8_NONE):
    return _product_workspace(lib().fq_glu_bwd_workspace_size(rows, k, n, experts, x_f8), device)


def _weights(w, offsets):
    """(experts, columns) of a weight; experts is 0 for one product."""
    if w.dim() != (2 if offsets is None else 3):
        raise ValueError("w must be [k, columns], or [experts, k, columns] with offsets")
    return (0 if offsets is None else w.shape[0]), w.shape[-1]


def fq_linear_fwd(x, w, bias=None, res=None, act: int = FQ_ACT_NONE, offsets=None, pre=None,
                  pre_f8: int = FQ_F8_NONE, pre_scales=None, y=None, ws=None, stream=None):
    """y = act(x @ w + bias) + res.

    x BF16 [rows, k], w BF16 [k, n]; with offsets (int32 [experts + 1], of
    fq_moe_sort) w [experts, k, n] and every segment of rows meets its own expert.
    y is BF16 unless it or res says FP32; y may be res.  pre, if given, receives
    the values before the activation for the backward: BF16 [rows, n], or uint8
    codes and pre_scales [rows, n / 32] with pre_f8=FQ_F8_MX.  Returns y."""
    if y is None or ws is None:
        torch = _torch()
        rows, k = _matrix(x, "x")
        experts, n = _weights(w, offsets)
        with _allocating(stream):
            if y is None:
                y = (torch.empty((rows, n), dtype=torch.bfloat16, device=x.device) if res is None
                     else torch.empty_like(res))
            if ws is None:
                ws = linear_fwd_workspace(rows, k, n, experts, x.device)
    st = (_binding_module or _binding()).linear_fwd(x, w, bias, res, offsets, act, pre, pre_f8,
                                                    pre_scales, y, ws, stream)
    if st:
        _check(st)
    return y


def _bwd_outputs(x, w, offsets, dx, dw, dbias, ws, need, dw_dtype, x_f8, workspace, halves, stream):
    """The outputs and the workspace of a product's backward that were not given."""
    need_dx, need_dw, need_dbias = need
    dx, dw, dbias = (v if n else None for v, n in zip((dx, dw, dbias), need))
    if (need_dx and dx is None) or (need_dw and dw is None) or (need_dbias and dbias is None) or ws is None:
        torch = _torch()
        rows, k = _matrix(x, "x")
        experts, cols = _weights(w, offsets)
        with _allocating(stream):
            if need_dx and dx is None:
                dx = torch.empty((rows, k), dtype=torch.bfloat16, device=x.device)
            if need_dw and dw is None:
                dw = torch.empty(w.shape, dtype=dw_dtype or torch.bfloat16, device=x.device)
            if need_dbias and dbias is None:
                dbias = torch.empty((*w.shape[:-2], cols), dtype=torch.float32, device=x.device)
            if ws is None:
                ws = workspace(rows, k, cols // halves, experts, x.device, x_f8)
    return dx, dw, dbias, ws


def fq_linear_bwd(dy, x, w, pre=None, act: int = FQ_ACT_NONE, offsets=None, x_f8: int = FQ_F8_NONE,
                  x_scales=None, pre_f8: int = FQ_F8_NONE, pre_scales=None, dx=None, dw=None,
                  dbias=None, ws=None, need_dx: bool = True, need_dw: bool = True,
                  need_dbias: bool = True, dw_dtype=None, stream=None):
    """(dx, dw, dbias) of fq_linear_fwd for the gradient dy of y (dy is also the
    gradient of its residual).  x BF16, or the codes of 8-bit rows with x_f8 and
    x_scales; pre what the forward kept, needed with an activation.  dw is BF16
    unless it or dw_dtype says FP32; need_...=False leaves an output out (None)."""
    dx, dw, dbias, ws = _bwd_outputs(x, w, offsets, dx, dw, dbias, ws, (need_dx, need_dw, need_dbias),
                                     dw_dtype, x_f8, linear_bwd_workspace, 1, stream)
    st = (_binding_module or _binding()).linear_bwd(dy, x, w, pre, x_f8, x_scales, pre_f8, pre_scales,
                                                    offsets, dx, dw, dbias, ws, act, stream)
    if st:
        _check(st)
    return dx, dw, dbias


def fq_glu_fwd(x, w, bias=None, act: int = FQ_ACT_SILU, alpha: float = 1.0, limit: float = math.inf,
               shift: float = 0.0, offsets=None, pre=None, pre_f8: int = FQ_F8_NONE, pre_scales=None,
               h=None, ws=None, stream=None):
    """h = act(min(g, limit)) * (clamp(u, -limit, limit) + shift) of [g, u] = x @ w + bias.

    x BF16 [rows, k], w BF16 [k, 2 n] (the gate's columns first), or [experts, k,
    2 n] with offsets; alpha is SiLU's slope.  pre as for fq_linear_fwd, of both
    projections: [rows, 2 n].  Returns h, BF16 [rows, n]."""
    if h is None or ws is None:
        torch = _torch()
        rows, k = _matrix(x, "x")
        experts, cols = _weights(w, offsets)
        with _allocating(stream):
            if h is None:
                h = torch.empty((rows, cols // 2), dtype=torch.bfloat16, device=x.device)
            if ws is None:
                ws = glu_fwd_workspace(rows, k, cols // 2, experts, x.device)
    st = (_binding_module or _binding()).glu_fwd(x, w, bias, offsets, act, alpha, limit, shift, pre,
                                                 pre_f8, pre_scales, h, ws, stream)
    if st:
        _check(st)
    return h


def fq_glu_bwd(dh, x, w, pre, act: int = FQ_ACT_SILU, alpha: float = 1.0, limit: float = math.inf,
               shift: float = 0.0, offsets=None, x_f8: int = FQ_F8_NONE, x_scales=None,
               pre_f8: int = FQ_F8_NONE, pre_scales=None, dx=None, dw=None, dbias=None, h=None, ws=None,
               need_dx: bool = True, need_dw: bool = True, need_dbias: bool = True, dw_dtype=None,
               stream=None):
    """(dx, dw, dbias) of fq_glu_fwd for the gradient dh of h, from what it kept.
    h, if given, receives the block's output again, for the next product's
    backward.  Other arguments as for fq_linear_bwd."""
    dx, dw, dbias, ws = _bwd_outputs(x, w, offsets, dx, dw, dbias, ws, (need_dx, need_dw, need_dbias),
                                     dw_dtype, x_f8, glu_bwd_workspace, 2, stream)
    st = (_binding_module or _binding()).glu_bwd(dh, x, w, pre, x_f8, x_scales, pre_f8, pre_scales,
                                                 offsets, dx, dw, dbias, ws, act, alpha, limit, shift, h,
                                                 stream)
    if st:
        _check(st)
    return dx, dw, dbias


def version() -> str:
    return lib().fq_version().decode()
