"""Python binding of libkq.so, the KroQuant MXFP4 activation quantizer for MI355X.

Argument marshalling only: every computation runs in the HIP kernels of
libkq.so (include/kq.h documents the C ABI). PyTorch provides device memory
and streams. There is no CPU fallback: if the library is missing or the
device is not a GPU, the calls raise.

Method: KroQuant (arXiv 2607.21446v1), Sec. 3.1-3.2 and 3.5 (Eq. 1, 4, 5, 12),
with the MXFP4 format of Sec. 4.1 / Appendix D.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkq.so")

KQ_OK, KQ_ERR_NULL, KQ_ERR_SHAPE, KQ_ERR_ALIGN, KQ_ERR_HIP, KQ_ERR_UNSUPPORTED = range(6)

# Every symbol include/kq.h declares.
EXPORTS = (
    "kq_quantize_mxfp4",
    "kq_transform_quantize_mxfp4",
    "kq_transform_quantize_mxfp4_form",
    "kq_smoothquant_quantize_mxfp4",
    "kq_quantize_mxfp4_f32",
    "kq_inverse_fold_weights",
    "kq_mxfp4_gemm",
    "kq_mxfp4_gemm_wide",
    "kq_pack_mxfp4_scales",
    "kq_lowrank_project_bf16",
    "kq_lowrank_project_bf16_split",
    "kq_lowrank_project_split",
    "kq_dequantize_mxfp4_bf16",
    "kq_mxfp4_gemm_packed",
    "kq_mxfp4_gemm_packed_bf16",
    "kq_mxfp4_gemm_packed_lowrank",
    "kq_mxfp4_gemm_packed_lowrank_split",
    "kq_transform_quantize_mxfp4_gemm",
    "kq_hadamard_quantize_mxfp4",
    "kq_transform_quantize_mxfp4_y16",
    "kq_transform_quantize_mxfp4_packed",
    "kq_lowrank_project",
    "kq_mxfp4_gemm_lowrank",
    "kq_gemm_f32",
    "kq_calib_workspace_bytes",
    "kq_calib_init",
    "kq_calib_step",
    "kq_calib_step_noalloc",
    "kq_layernorm",
    "kq_layernorm_backward_workspace_bytes",
    "kq_layernorm_backward",
    "kq_layernorm_quantize_mxfp4",
    "kq_mxfp4_linear",
    "kq_mxfp4_linear_backward_workspace_bytes",
    "kq_mxfp4_linear_backward",
    "kq_mxfp4_gated_linear",
    "kq_mxfp4_gated_linear_backward_workspace_bytes",
    "kq_mxfp4_gated_linear_backward",
    "kq_rope_frequencies",
    "kq_headnorm_rope",
    "kq_headnorm_rope_backward_workspace_bytes",
    "kq_headnorm_rope_backward",
    "kq_cache_write_mxfp4",
    "kq_cache_read_mxfp4",
    "kq_status_string",
    "kq_last_hip_error",
    "kq_factors_from_lu",
)

_lib = None


class KQError(RuntimeError):
    def __init__(self, fn, status, lib):
        msg = lib.kq_status_string(status).decode()
        if status == KQ_ERR_HIP:
            msg += " (hipError_t %d)" % lib.kq_last_hip_error()
        super().__init__("%s: %s" % (fn, msg))
        self.status = status


def lib():
    """Load libkq.so (built by ``__graft_entry__.build()`` or ``python -m ...build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkq.so is not built: run `python -m mxfp4_activation_quantizer_amd.build`")
        # torch's HIP runtime first, so that libkq.so is bound to it: the other way round the process would have two, and
        # libkq.so's would see no device
        try:
            _torch()
        except ImportError:  # the host's helpers need none
            pass
        L = ctypes.CDLL(LIB_PATH)
        p, i64, st, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
        for name, args in {
            "kq_quantize_mxfp4": [p, i64, i64, i64, p, p, p],
            "kq_transform_quantize_mxfp4": [p, i64, i64, i64, p, p, p, p, p],
            "kq_transform_quantize_mxfp4_form": [p, i64, i64, i64, p, p, p, p, st, p],
            "kq_smoothquant_quantize_mxfp4": [p, i64, i64, i64, p, p, p, p],
            "kq_quantize_mxfp4_f32": [p, i64, i64, i64, p, p, p],
            "kq_inverse_fold_weights": [p, i64, i64, p, p, p],
            "kq_factors_from_lu": [p, i64, p],
            "kq_mxfp4_gemm": [p, p, p, p, i64, i64, i64, p, i64, p],
            "kq_mxfp4_gemm_wide": [p, p, p, p, i64, i64, i64, p, i64, p],
            "kq_pack_mxfp4_scales": [p, i64, i64, p, p],
            "kq_lowrank_project_bf16": [p, i64, i64, i64, p, i64, p, p],
            "kq_lowrank_project_bf16_split": [p, i64, i64, i64, p, i64, p, p, p],
            "kq_lowrank_project_split": [p, i64, i64, i64, p, p, i64, p, p, p],
            "kq_dequantize_mxfp4_bf16": [p, p, i64, i64, p, p],
            "kq_mxfp4_gemm_packed": [p, p, p, p, i64, i64, i64, p, i64, p],
            "kq_mxfp4_gemm_packed_bf16": [p, p, p, p, i64, i64, i64, p, i64, p],
            "kq_mxfp4_gemm_packed_lowrank": [p, p, p, p, i64, i64, i64, p, p, p, i64, p, i64, p],
            "kq_mxfp4_gemm_packed_lowrank_split": [p, p, p, p, i64, i64, i64, p, p, p, i64, p, i64, p],
            "kq_transform_quantize_mxfp4_gemm": [p, i64, i64, i64, p, p, p, i64, p, i64, p],
            "kq_hadamard_quantize_mxfp4": [p, i64, i64, i64, i64, p, p, p, p],
            "kq_transform_quantize_mxfp4_y16": [p, i64, i64, i64, p, p, p, p, p],
            "kq_transform_quantize_mxfp4_packed": [p, i64, i64, i64, p, p, p, p, p],
            "kq_lowrank_project": [p, i64, i64, i64, p, p, i64, p, p],
            "kq_mxfp4_gemm_lowrank": [p, p, p, p, i64, i64, i64, p, p, p, i64, p, i64, p],
            "kq_gemm_f32": [st, st, i64, i64, i64, ctypes.c_float, p, i64, p, i64, ctypes.c_float, p, i64, p,
                            i64, p],
            "kq_calib_workspace_bytes": [i64, i64, i64, p],
            "kq_calib_init": [p, i64, i64, p, i64, p, i64, p],
            "kq_calib_step": [p, i64, i64, i64, p, p, p, i64, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                              ctypes.c_float, p, st, p, p, p, i64, p],
            "kq_calib_step_noalloc": [p, p, i64, i64, i64, p, p, p, i64, ctypes.c_float, ctypes.c_float,
                                      ctypes.c_float, ctypes.c_float, p, st, p, p, p],
            "kq_layernorm": [p, st, i64, i64, i64, p, p, ctypes.c_float, p, i64, p, p, p],
            "kq_layernorm_backward_workspace_bytes": [i64, i64, p],
            "kq_layernorm_backward": [p, i64, p, i64, st, i64, i64, p, p, p, p, i64, p, p, p, i64, p],
            "kq_layernorm_quantize_mxfp4": [p, st, i64, i64, i64, p, p, ctypes.c_float, p, p, p, st, p, p, p, p],
            "kq_mxfp4_linear": [p, p, p, p, st, i64, i64, i64, p, st, st, p, i64, p, i64, p, i64, p],
            "kq_mxfp4_linear_backward_workspace_bytes": [i64, i64, p],
            "kq_mxfp4_linear_backward": [p, i64, p, i64, st, i64, i64, st, p, i64, p, p, i64, p],
            "kq_mxfp4_gated_linear": [p, p, p, p, p, p, st, i64, i64, i64, p, p, st, st, p, i64, p, i64, p, i64, p],
            "kq_mxfp4_gated_linear_backward_workspace_bytes": [i64, i64, p],
            "kq_mxfp4_gated_linear_backward": [p, i64, p, i64, p, i64, st, i64, i64, st, p, i64, p, i64, p, p, p, i64, p],
            "kq_rope_frequencies": [i64, f64, st, f64, f64, f64, f64, p],
            "kq_headnorm_rope": [p, st, i64, i64, i64, i64, i64, st, p, p, i64, ctypes.c_float, p, p, i64, i64, p],
            "kq_headnorm_rope_backward_workspace_bytes": [i64, i64, p],
            "kq_headnorm_rope_backward": [p, i64, i64, p, i64, i64, st, i64, i64, i64, st, p, p, i64, ctypes.c_float,
                                          p, p, i64, i64, p, p, p, i64, p],
            "kq_cache_write_mxfp4": [p, i64, i64, i64, p, i64, i64, i64, st, i64, i64, st, p, ctypes.c_float, p, p,
                                     i64, p, p, p, p, p],
            "kq_cache_read_mxfp4": [p, i64, p, p, i64, i64, i64, st, p, i64, i64, p],
        }.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = st
        L.kq_status_string.argtypes = [st]
        L.kq_status_string.restype = ctypes.c_char_p
        L.kq_last_hip_error.argtypes = []
        L.kq_last_hip_error.restype = st
        _lib = L
    return _lib


def _check(fn, status):
    if status != KQ_OK:
        raise KQError(fn, status, lib())


def _torch():
    import torch
    return torch


def _stream_ptr(stream):
    if stream is None:
        return ctypes.c_void_p(_current_stream(_torch().cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name, dtypes):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    return t


def _rows(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("%s must be 2-D with unit column stride" % name)
    return t.shape[0], t.shape[1], t.stride(0)


def _p(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _outputs(m, d, device, codes, scales):
    torch = _torch()
    if codes is None:
        codes = torch.empty((m, d // 2), dtype=torch.uint8, device=device)
    if scales is None:
        scales = torch.empty((m, d // 32), dtype=torch.uint8, device=device)
    _dev(codes, "codes", (torch.uint8,))
    _dev(scales, "scales", (torch.uint8,))
    if tuple(codes.shape) != (m, d // 2) or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous [m][d/2] uint8 tensor")
    if tuple(scales.shape) != (m, d // 32) or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous [m][d/32] uint8 tensor")
    return codes, scales


def _bf16_input(A):
    torch = _torch()
    _dev(A, "A", (torch.bfloat16, torch.int16, torch.uint16))
    return _rows(A, "A")


def quantize_mxfp4(A, codes=None, scales=None, stream=None):
    """MXFP4 codes [m][d/2] and E8M0 scales [m][d/32] of bf16 A [m][d] (T = I)."""
    m, d, lda = _bf16_input(A)
    codes, scales = _outputs(m, d, A.device, codes, scales)
    _check("kq_quantize_mxfp4",
           lib().kq_quantize_mxfp4(_p(A), m, d, lda, _p(codes), _p(scales), _stream_ptr(stream)))
    return codes, scales


FORMS = {"butterfly": 0, "mfma": 1, "mfma_lds": 2}  # kq_transform_form


def transform_quantize_mxfp4(A, factors, codes=None, scales=None, y_debug=None, stream=None, form=None):
    """Fused y = A T (per-block Kronecker factors fp32 [d/32][5][2][2]) then MXFP4.

    ``y_debug``: optional fp32 [m][d] tensor that receives y (check mode).
    ``form``: None (the library's default, the butterfly form) or one of FORMS.
    """
    torch = _torch()
    m, d, lda = _bf16_input(A)
    _dev(factors, "factors", (torch.float32,))
    if factors.numel() != (d // 32) * 20 or not factors.is_contiguous():
        raise ValueError("factors must be contiguous fp32 [d/32][5][2][2]")
    if y_debug is not None:
        _dev(y_debug, "y_debug", (torch.float32,))
        if tuple(y_debug.shape) != (m, d) or not y_debug.is_contiguous():
            raise ValueError("y_debug must be a contiguous fp32 [m][d] tensor")
    codes, scales = _outputs(m, d, A.device, codes, scales)
    if form is None:
        _check("kq_transform_quantize_mxfp4",
               lib().kq_transform_quantize_mxfp4(_p(A), m, d, lda, _p(factors), _p(codes), _p(scales),
                                                 _p(y_debug), _stream_ptr(stream)))
    else:
        _check("kq_transform_quantize_mxfp4_form",
               lib().kq_transform_quantize_mxfp4_form(_p(A), m, d, lda, _p(factors), _p(codes), _p(scales),
                                                      _p(y_debug), FORMS[form], _stream_ptr(stream)))
    return codes, scales


def hadamard_quantize_mxfp4(A, n, codes=None, scales=None, y_debug=None, stream=None):
    """Block-Hadamard baseline: each group of n channels times H_n / sqrt(n), then MXFP4.

    n = 32 is the block-size Hadamard, n = d the full-width transform (FWHT).
    """
    torch = _torch()
    m, d, lda = _bf16_input(A)
    if y_debug is not None:
        _dev(y_debug, "y_debug", (torch.float32,))
        if tuple(y_debug.shape) != (m, d) or not y_debug.is_contiguous():
            raise ValueError("y_debug must be a contiguous fp32 [m][d] tensor")
    codes, scales = _outputs(m, d, A.device, codes, scales)
    _check("kq_hadamard_quantize_mxfp4",
           lib().kq_hadamard_quantize_mxfp4(_p(A), m, d, lda, int(n), _p(codes), _p(scales),
                                            _p(y_debug), _stream_ptr(stream)))
    return codes, scales


def transform_quantize_mxfp4_y16(A, factors, codes=None, scales=None, y16=None, stream=None):
    """Fused y = A T then MXFP4, also writing bf16(y) [m][d] (the 16-bit activation the
    low-rank branch of Eq. 11 consumes). Returns codes, scales, y16."""
    torch = _torch()
    m, d, lda = _bf16_input(A)
    _dev(factors, "factors", (torch.float32,))
    if factors.numel() != (d // 32) * 20 or not factors.is_contiguous():
        raise ValueError("factors must be contiguous fp32 [d/32][5][2][2]")
    if y16 is None:
        y16 = torch.empty((m, d), dtype=torch.bfloat16, device=A.device)
    _dev(y16, "y16", (torch.bfloat16,))
    if tuple(y16.shape) != (m, d) or not y16.is_contiguous():
        raise ValueError("y16 must be a contiguous bf16 [m][d] tensor")
    codes, scales = _outputs(m, d, A.device, codes, scales)
    _check("kq_transform_quantize_mxfp4_y16",
           lib().kq_transform_quantize_mxfp4_y16(_p(A), m, d, lda, _p(factors), _p(codes), _p(scales), _p(y16),
                                                 _stream_ptr(stream)))
    return codes, scales, y16


def transform_quantize_mxfp4_packed(A, factors, codes=None, packed_scales=None, y16=None, want_y16=False,
                                     stream=None):
    """Fused y = A T then MXFP4 with the scales written in the packed-GEMM layout
    [d/256][m][8] (what pack_mxfp4_scales makes of them; d % 256 == 0), optionally also
    bf16(y) [m][d] (y16, or want_y16=True to allocate it). Returns codes, packed scales, y16
    (or None)."""
    torch = _torch()
    m, d, lda = _bf16_input(A)
    _dev(factors, "factors", (torch.float32,))
    if factors.numel() != (d // 32) * 20 or not factors.is_contiguous():
        raise ValueError("factors must be contiguous fp32 [d/32][5][2][2]")
    if codes is None:
        codes = torch.empty((m, d // 2), dtype=torch.uint8, device=A.device)
    _dev(codes, "codes", (torch.uint8,))
    if tuple(codes.shape) != (m, d // 2) or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous [m][d/2] uint8 tensor")
    if packed_scales is None:
        packed_scales = torch.empty((d // 256 if d % 256 == 0 else 0, m, 8), dtype=torch.uint8, device=A.device)
    _dev(packed_scales, "packed_scales", (torch.uint8,))
    if packed_scales.numel() != m * (d // 32) or not packed_scales.is_contiguous():
        raise ValueError("packed_scales must be a contiguous uint8 tensor of m * d/32 bytes")
    if y16 is None and want_y16:
        y16 = torch.empty((m, d), dtype=torch.bfloat16, device=A.device)
    if y16 is not None:
        _dev(y16, "y16", (torch.bfloat16,))
        if tuple(y16.shape) != (m, d) or not y16.is_contiguous():
            raise ValueError("y16 must be a contiguous bf16 [m][d] tensor")
    _check("kq_transform_quantize_mxfp4_packed",
           lib().kq_transform_quantize_mxfp4_packed(_p(A), m, d, lda, _p(factors), _p(codes), _p(packed_scales),
                                                    _p(y16) if y16 is not None else None, _stream_ptr(stream)))
    return codes, packed_scales, y16


def lowrank_project(X16, codes_r, scales_r, out=None, stream=None):
    """Z = X16 Q(R)^T in fp32: X16 bf16 [m][d], R in MXFP4 (codes [r][d/2], scales [r][d/32])."""
    torch = _torch()
    _dev(X16, "X16", (torch.bfloat16, torch.int16, torch.uint16))
    m, d, ldx = _rows(X16, "X16")
    for t, nm in ((codes_r, "codes_r"), (scales_r, "scales_r")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    r = codes_r.shape[0]
    if tuple(codes_r.shape) != (r, d // 2) or tuple(scales_r.shape) != (r, d // 32):
        raise ValueError("R operand shapes do not match X16")
    if out is None:
        out = torch.empty((m, r), dtype=torch.float32, device=X16.device)
    _dev(out, "out", (torch.float32,))
    if tuple(out.shape) != (m, r) or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [m][r] tensor")
    _check("kq_lowrank_project",
           lib().kq_lowrank_project(_p(X16), m, d, ldx, _p(codes_r), _p(scales_r), r, _p(out), _stream_ptr(stream)))
    return out


def lowrank_project_split(X16, codes_r, scales_r, Zh=None, Zl=None, stream=None):
    """As lowrank_project (R in MXFP4), Z written as its bf16 split: Zh = bf16(Z),
    Zl = bf16(Z - Zh) (bf16 [m][r] each). Returns Zh, Zl."""
    torch = _torch()
    _dev(X16, "X16", (torch.bfloat16, torch.int16, torch.uint16))
    m, d, ldx = _rows(X16, "X16")
    for t, nm in ((codes_r, "codes_r"), (scales_r, "scales_r")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    r = codes_r.shape[0]
    if tuple(codes_r.shape) != (r, d // 2) or tuple(scales_r.shape) != (r, d // 32):
        raise ValueError("R operand shapes do not match X16")
    outs = []
    for t, nm in ((Zh, "Zh"), (Zl, "Zl")):
        if t is None:
            t = torch.empty((m, r), dtype=torch.bfloat16, device=X16.device)
        _dev(t, nm, (torch.bfloat16,))
        if tuple(t.shape) != (m, r) or not t.is_contiguous():
            raise ValueError(nm + " must be a contiguous bf16 [m][r] tensor")
        outs.append(t)
    Zh, Zl = outs
    _check("kq_lowrank_project_split",
           lib().kq_lowrank_project_split(_p(X16), m, d, ldx, _p(codes_r), _p(scales_r), r, _p(Zh), _p(Zl),
                                          _stream_ptr(stream)))
    return Zh, Zl


def dequantize_mxfp4_bf16(codes, scales, out=None, stream=None):
    """deq(codes, scales) as bf16 [rows][k] (exact): codes [rows][k/2], scales [rows][k/32]."""
    torch = _torch()
    for t, nm in ((codes, "codes"), (scales, "scales")):
        _dev(t, nm, (torch.uint8,))
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(nm + " must be a contiguous 2-D uint8 tensor")
    rows, kb = codes.shape
    k = kb * 2
    if tuple(scales.shape) != (rows, k // 32):
        raise ValueError("scales must be [rows][k/32]")
    if out is None:
        out = torch.empty((rows, k), dtype=torch.bfloat16, device=codes.device)
    _dev(out, "out", (torch.bfloat16, torch.int16, torch.uint16))
    if tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 [rows][k] tensor")
    _check("kq_dequantize_mxfp4_bf16",
           lib().kq_dequantize_mxfp4_bf16(_p(codes), _p(scales), rows, k, _p(out), _stream_ptr(stream)))
    return out


def lowrank_project_bf16(X16, R16, out=None, stream=None):
    """Z = X16 R16^T in fp32: X16 bf16 [m][d], R16 bf16 [r][d] (e.g. dequantize_mxfp4_bf16 of R)."""
    torch = _torch()
    _dev(X16, "X16", (torch.bfloat16, torch.int16, torch.uint16))
    _dev(R16, "R16", (torch.bfloat16, torch.int16, torch.uint16))
    m, d, ldx = _rows(X16, "X16")
    if R16.dim() != 2 or R16.shape[1] != d or not R16.is_contiguous():
        raise ValueError("R16 must be a contiguous bf16 [r][d] tensor")
    r = R16.shape[0]
    if out is None:
        out = torch.empty((m, r), dtype=torch.float32, device=X16.device)
    _dev(out, "out", (torch.float32,))
    if tuple(out.shape) != (m, r) or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [m][r] tensor")
    _check("kq_lowrank_project_bf16",
           lib().kq_lowrank_project_bf16(_p(X16), m, d, ldx, _p(R16), r, _p(out), _stream_ptr(stream)))
    return out


def lowrank_project_bf16_split(X16, R16, Zh=None, Zl=None, stream=None):
    """As lowrank_project_bf16, Z written as its bf16 split: Zh = bf16(Z), Zl = bf16(Z - Zh)
    (bf16 [m][r] each). Returns Zh, Zl."""
    torch = _torch()
    _dev(X16, "X16", (torch.bfloat16, torch.int16, torch.uint16))
    _dev(R16, "R16", (torch.bfloat16, torch.int16, torch.uint16))
    m, d, ldx = _rows(X16, "X16")
    if R16.dim() != 2 or R16.shape[1] != d or not R16.is_contiguous():
        raise ValueError("R16 must be a contiguous bf16 [r][d] tensor")
    r = R16.shape[0]
    outs = []
    for t, nm in ((Zh, "Zh"), (Zl, "Zl")):
        if t is None:
            t = torch.empty((m, r), dtype=torch.bfloat16, device=X16.device)
        _dev(t, nm, (torch.bfloat16,))
        if tuple(t.shape) != (m, r) or not t.is_contiguous():
            raise ValueError(nm + " must be a contiguous bf16 [m][r] tensor")
        outs.append(t)
    Zh, Zl = outs
    _check("kq_lowrank_project_bf16_split",
           lib().kq_lowrank_project_bf16_split(_p(X16), m, d, ldx, _p(R16), r, _p(Zh), _p(Zl), _stream_ptr(stream)))
    return Zh, Zl


def mxfp4_gemm_lowrank(codes_a, scales_a, codes_w, scales_w, Z, codes_l, scales_l, out=None, stream=None):
    """O = deq(A) deq(W)^T + Z deq(L)^T (Eq. 11's two terms): Z fp32 [m][r], L in MXFP4
    (codes [n][r/2], scales [n][r/32])."""
    torch = _torch()
    for t, nm in ((codes_a, "codes_a"), (scales_a, "scales_a"), (codes_w, "codes_w"), (scales_w, "scales_w"),
                  (codes_l, "codes_l"), (scales_l, "scales_l")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    _dev(Z, "Z", (torch.float32,))
    m, kb = codes_a.shape
    n = codes_w.shape[0]
    k = kb * 2
    r = Z.shape[1]
    if tuple(codes_w.shape) != (n, kb) or tuple(scales_a.shape) != (m, k // 32) or \
            tuple(scales_w.shape) != (n, k // 32) or Z.shape[0] != m or not Z.is_contiguous() or \
            tuple(codes_l.shape) != (n, r // 2) or tuple(scales_l.shape) != (n, r // 32):
        raise ValueError("operand shapes do not match")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=codes_a.device)
    _dev(out, "out", (torch.float32,))
    if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or out.stride(1) != 1:
        raise ValueError("out must be fp32 [m][n] with unit column stride")
    _check("kq_mxfp4_gemm_lowrank",
           lib().kq_mxfp4_gemm_lowrank(_p(codes_a), _p(scales_a), _p(codes_w), _p(scales_w), m, n, k, _p(Z),
                                       _p(codes_l), _p(scales_l), r, _p(out), out.stride(0), _stream_ptr(stream)))
    return out


def smoothquant_quantize_mxfp4(A, inv_scale, codes=None, scales=None, stream=None):
    """SmoothQuant baseline: y_c = fl32(a_c * inv_scale[c]) then MXFP4."""
    torch = _torch()
    m, d, lda = _bf16_input(A)
    _dev(inv_scale, "inv_scale", (torch.float32,))
    if inv_scale.numel() < d or not inv_scale.is_contiguous():
        raise ValueError("inv_scale must be a contiguous fp32 vector of length d")
    codes, scales = _outputs(m, d, A.device, codes, scales)
    _check("kq_smoothquant_quantize_mxfp4",
           lib().kq_smoothquant_quantize_mxfp4(_p(A), m, d, lda, _p(inv_scale), _p(codes),
                                               _p(scales), _stream_ptr(stream)))
    return codes, scales


def quantize_mxfp4_f32(X, codes=None, scales=None, stream=None):
    """MXFP4 codes and scales of fp32 X [m][d]."""
    torch = _torch()
    _dev(X, "X", (torch.float32,))
    m, d, ldx = _rows(X, "X")
    codes, scales = _outputs(m, d, X.device, codes, scales)
    _check("kq_quantize_mxfp4_f32",
           lib().kq_quantize_mxfp4_f32(_p(X), m, d, ldx, _p(codes), _p(scales), _stream_ptr(stream)))
    return codes, scales


def inverse_fold_weights(W, factors, out=None, stream=None):
    """W' = W T^{-T} for fp32 W [o][d] (the weight side of Eq. 1)."""
    torch = _torch()
    _dev(W, "W", (torch.float32,))
    _dev(factors, "factors", (torch.float32,))
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    o, d = W.shape
    if factors.numel() != (d // 32) * 20 or not factors.is_contiguous():
        raise ValueError("factors must be contiguous fp32 [d/32][5][2][2]")
    if out is None:
        out = torch.empty_like(W)
    _dev(out, "out", (torch.float32,))
    if out.shape != W.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 tensor shaped like W")
    _check("kq_inverse_fold_weights",
           lib().kq_inverse_fold_weights(_p(W), o, d, _p(factors), _p(out), _stream_ptr(stream)))
    return out


def _gemm_operands(codes_a, scales_a, codes_w, scales_w, out):
    torch = _torch()
    for t, nm in ((codes_a, "codes_a"), (scales_a, "scales_a"), (codes_w, "codes_w"), (scales_w, "scales_w")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    m, kb = codes_a.shape
    n = codes_w.shape[0]
    k = kb * 2
    if tuple(codes_w.shape) != (n, kb) or tuple(scales_a.shape) != (m, k // 32) or \
            tuple(scales_w.shape) != (n, k // 32):
        raise ValueError("operand shapes do not match")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=codes_a.device)
    _dev(out, "out", (torch.float32,))
    if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or out.stride(1) != 1:
        raise ValueError("out must be fp32 [m][n] with unit column stride")
    return m, n, k, out


def mxfp4_gemm(codes_a, scales_a, codes_w, scales_w, out=None, stream=None):
    """O = deq(A) deq(W)^T in fp32 from MXFP4 operands (codes [rows][k/2], scales [rows][k/32])."""
    m, n, k, out = _gemm_operands(codes_a, scales_a, codes_w, scales_w, out)
    _check("kq_mxfp4_gemm",
           lib().kq_mxfp4_gemm(_p(codes_a), _p(scales_a), _p(codes_w), _p(scales_w), m, n, k, _p(out),
                               out.stride(0), _stream_ptr(stream)))
    return out


def pack_mxfp4_scales(scales, out=None, stream=None):
    """MXFP4 scales [rows][k/32] -> the GEMM-ready layout [k/256][rows][8] (k % 256 == 0)."""
    torch = _torch()
    _dev(scales, "scales", (torch.uint8,))
    if scales.dim() != 2 or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous [rows][k/32] uint8 tensor")
    rows, kb = scales.shape
    k = kb * 32
    if out is None:
        out = torch.empty((kb // 8 if kb % 8 == 0 else 0, rows, 8), dtype=torch.uint8, device=scales.device)
    _dev(out, "out", (torch.uint8,))
    if out.numel() != rows * kb or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor of rows * k/32 bytes")
    _check("kq_pack_mxfp4_scales",
           lib().kq_pack_mxfp4_scales(_p(scales), rows, k, _p(out), _stream_ptr(stream)))
    return out


def mxfp4_gemm_packed(codes_a, packed_scales_a, codes_w, packed_scales_w, out=None, stream=None, bf16=False):
    """O = deq(A) deq(W)^T in fp32 (bf16=True: rounded to bf16, half the output bytes), scales
    packed by pack_mxfp4_scales (k % 256 == 0)."""
    torch = _torch()
    for t, nm in ((codes_a, "codes_a"), (packed_scales_a, "packed_scales_a"), (codes_w, "codes_w"),
                  (packed_scales_w, "packed_scales_w")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    m, kb = codes_a.shape
    n = codes_w.shape[0]
    k = kb * 2
    if tuple(codes_w.shape) != (n, kb) or packed_scales_a.numel() != m * (k // 32) or \
            packed_scales_w.numel() != n * (k // 32):
        raise ValueError("operand shapes do not match")
    odt = torch.bfloat16 if bf16 else torch.float32
    if out is None:
        out = torch.empty((m, n), dtype=odt, device=codes_a.device)
    _dev(out, "out", (odt,))
    if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or out.stride(1) != 1:
        raise ValueError("out must be %s [m][n] with unit column stride" % ("bf16" if bf16 else "fp32"))
    name = "kq_mxfp4_gemm_packed_bf16" if bf16 else "kq_mxfp4_gemm_packed"
    _check(name, getattr(lib(), name)(_p(codes_a), _p(packed_scales_a), _p(codes_w), _p(packed_scales_w), m, n, k,
                                      _p(out), out.stride(0), _stream_ptr(stream)))
    return out


def mxfp4_gemm_packed_lowrank(codes_a, packed_scales_a, codes_w, packed_scales_w, Z, codes_l, scales_l, out=None,
                              stream=None):
    """O = deq(A) deq(W)^T + Z deq(L)^T on the packed-scale GEMM (k % 256 == 0): Z fp32 [m][r],
    L in MXFP4 (codes [n][r/2], scales [n][r/32])."""
    torch = _torch()
    for t, nm in ((codes_a, "codes_a"), (packed_scales_a, "packed_scales_a"), (codes_w, "codes_w"),
                  (packed_scales_w, "packed_scales_w"), (codes_l, "codes_l"), (scales_l, "scales_l")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    _dev(Z, "Z", (torch.float32,))
    m, kb = codes_a.shape
    n = codes_w.shape[0]
    k = kb * 2
    r = Z.shape[1] if Z.dim() == 2 else -1
    if tuple(codes_w.shape) != (n, kb) or packed_scales_a.numel() != m * (k // 32) or \
            packed_scales_w.numel() != n * (k // 32) or tuple(Z.shape) != (m, r) or not Z.is_contiguous() or \
            tuple(codes_l.shape) != (n, r // 2) or tuple(scales_l.shape) != (n, r // 32):
        raise ValueError("operand shapes do not match")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=codes_a.device)
    _dev(out, "out", (torch.float32,))
    if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or out.stride(1) != 1:
        raise ValueError("out must be fp32 [m][n] with unit column stride")
    _check("kq_mxfp4_gemm_packed_lowrank",
           lib().kq_mxfp4_gemm_packed_lowrank(_p(codes_a), _p(packed_scales_a), _p(codes_w), _p(packed_scales_w), m,
                                              n, k, _p(Z), _p(codes_l), _p(scales_l), r, _p(out), out.stride(0),
                                              _stream_ptr(stream)))
    return out


def mxfp4_gemm_packed_lowrank_split(codes_a, packed_scales_a, codes_w, packed_scales_w, Zh, Zl, L16, out=None,
                                    stream=None):
    """mxfp4_gemm_packed_lowrank with the branch's operands prepared once: Z split as Zh, Zl
    (bf16 [m][r], lowrank_project_bf16_split) and deq(L) in bf16 [n][r]
    (dequantize_mxfp4_bf16 of L). Bit-identical to the fp32-Z form on the Z they split."""
    torch = _torch()
    for t, nm in ((codes_a, "codes_a"), (packed_scales_a, "packed_scales_a"), (codes_w, "codes_w"),
                  (packed_scales_w, "packed_scales_w")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    for t, nm in ((Zh, "Zh"), (Zl, "Zl"), (L16, "L16")):
        _dev(t, nm, (torch.bfloat16, torch.int16, torch.uint16))
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(nm + " must be a contiguous 2-d bf16 tensor")
    m, kb = codes_a.shape
    n = codes_w.shape[0]
    k = kb * 2
    r = Zh.shape[1]
    if tuple(codes_w.shape) != (n, kb) or packed_scales_a.numel() != m * (k // 32) or \
            packed_scales_w.numel() != n * (k // 32) or tuple(Zh.shape) != (m, r) or tuple(Zl.shape) != (m, r) or \
            tuple(L16.shape) != (n, r):
        raise ValueError("operand shapes do not match")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=codes_a.device)
    _dev(out, "out", (torch.float32,))
    if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or out.stride(1) != 1:
        raise ValueError("out must be fp32 [m][n] with unit column stride")
    _check("kq_mxfp4_gemm_packed_lowrank_split",
           lib().kq_mxfp4_gemm_packed_lowrank_split(_p(codes_a), _p(packed_scales_a), _p(codes_w),
                                                    _p(packed_scales_w), m, n, k, _p(Zh), _p(Zl), _p(L16), r,
                                                    _p(out), out.stride(0), _stream_ptr(stream)))
    return out


def mxfp4_gemm_wide(codes_a, scales_a, codes_w, scales_w, out=None, stream=None):
    """As mxfp4_gemm, on the 128 x 512-tile kernel (bit-identical results)."""
    torch = _torch()
    m, n, k, out = _gemm_operands(codes_a, scales_a, codes_w, scales_w, out)
    _check("kq_mxfp4_gemm_wide",
           lib().kq_mxfp4_gemm_wide(_p(codes_a), _p(scales_a), _p(codes_w), _p(scales_w), m, n, k, _p(out),
                                    out.stride(0), _stream_ptr(stream)))
    return out


def transform_quantize_mxfp4_gemm(A, factors, codes_w, scales_w, out=None, stream=None):
    """O = deq(Q(A T)) deq(W)^T in fp32: the Kronecker transform and MXFP4 quantizer of A
    (bf16 [m][k], factors fp32 [k/32][5][2][2]) run inside the W4A4 product with the MXFP4
    weights (codes [n][k/2], scales [n][k/32])."""
    torch = _torch()
    m, k, lda = _bf16_input(A)
    _dev(factors, "factors", (torch.float32,))
    if factors.numel() != (k // 32) * 20 or not factors.is_contiguous():
        raise ValueError("factors must be contiguous fp32 [k/32][5][2][2]")
    for t, nm in ((codes_w, "codes_w"), (scales_w, "scales_w")):
        _dev(t, nm, (torch.uint8,))
        if not t.is_contiguous():
            raise ValueError(nm + " must be contiguous")
    n = codes_w.shape[0]
    if tuple(codes_w.shape) != (n, k // 2) or tuple(scales_w.shape) != (n, k // 32):
        raise ValueError("weight operand shapes do not match A")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    _dev(out, "out", (torch.float32,))
    if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or out.stride(1) != 1:
        raise ValueError("out must be fp32 [m][n] with unit column stride")
    _check("kq_transform_quantize_mxfp4_gemm",
           lib().kq_transform_quantize_mxfp4_gemm(_p(A), m, k, lda, _p(factors), _p(codes_w), _p(scales_w), n,
                                                  _p(out), out.stride(0), _stream_ptr(stream)))
    return out


def gemm_f32(A, B, transa=False, transb=False, alpha=1.0, beta=0.0, C=None, out=None, stream=None):
    """D = alpha op(A) op(B) + beta C in fp32 (row-major operands)."""
    torch = _torch()
    for t, nm in ((A, "A"), (B, "B")):
        _dev(t, nm, (torch.float32,))
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(nm + " must be 2-D with unit column stride")
    m, k = (A.shape[1], A.shape[0]) if transa else (A.shape[0], A.shape[1])
    kb, n = (B.shape[1], B.shape[0]) if transb else (B.shape[0], B.shape[1])
    if kb != k:
        raise ValueError("inner dimensions do not match")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    _dev(out, "out", (torch.float32,))
    if tuple(out.shape) != (m, n) or out.stride(1) != 1:
        raise ValueError("out must be fp32 [m][n] with unit column stride")
    if beta != 0.0:
        _dev(C, "C", (torch.float32,))
        if tuple(C.shape) != (m, n) or C.stride(1) != 1 or C.stride(0) != out.stride(0):
            raise ValueError("C must be fp32 [m][n] with the row stride of out")
    _check("kq_gemm_f32",
           lib().kq_gemm_f32(int(transa), int(transb), m, n, k, float(alpha), _p(A), A.stride(0), _p(B),
                             B.stride(0), float(beta), _p(C) if beta != 0.0 else None, out.stride(0), _p(out),
                             out.stride(0), _stream_ptr(stream)))
    return out


class Calibration:
    """Layer-wise calibration of the Kronecker factors (Sec. 3.3) on one GPU.

    Holds the device state: the 15 parameters per block (a, b, c of Eq. 6 for
    each of the five factors), Adam's moments, the Eq. 10 weights and the
    workspace. Every computation runs in libkq.so (kq_calib_init / kq_calib_step).
    """

    def __init__(self, A, W, theta=None, stream=None):
        torch = _torch()
        _dev(A, "A", (torch.bfloat16, torch.int16, torch.uint16))
        _dev(W, "W", (torch.float32,))
        if not A.is_contiguous() or not W.is_contiguous() or A.dim() != 2 or W.dim() != 2:
            raise ValueError("A [M][d] and W [o][d] must be contiguous")
        self.M, self.d = A.shape
        self.o = W.shape[0]
        if W.shape[1] != self.d:
            raise ValueError("W must be [o][d]")
        self.W = W
        self.stream = stream
        nbytes = ctypes.c_int64(0)
        _check("kq_calib_workspace_bytes",
               lib().kq_calib_workspace_bytes(self.M, self.d, self.o, ctypes.byref(nbytes)))
        self.ws = torch.empty(nbytes.value + 256, dtype=torch.uint8, device=A.device)
        self._ws_ptr = (self.ws.data_ptr() + 255) // 256 * 256
        nblk = self.d // 32
        if theta is None:  # Hadamard initialization (Sec. 3.2): a = b = 1/sqrt(2), c = 1
            theta = torch.tensor([2.0 ** -0.5, 2.0 ** -0.5, 1.0], dtype=torch.float32).repeat(nblk, 5, 1)
        self.theta = theta.to(device=A.device, dtype=torch.float32).contiguous().clone()
        if self.theta.numel() != nblk * 15:
            raise ValueError("theta must hold 15 parameters per block")
        self.m = torch.zeros_like(self.theta)
        self.v = torch.zeros_like(self.theta)
        self.lambdas = torch.zeros(2, dtype=torch.float32, device=A.device)
        self.losses = torch.zeros(3, dtype=torch.float32, device=A.device)
        self.grad = torch.zeros_like(self.theta)
        self.t = 0
        _check("kq_calib_init",
               lib().kq_calib_init(_p(A), self.M, self.d, _p(W), self.o, ctypes.c_void_p(self._ws_ptr),
                                   self.ws.numel() - 256, _stream_ptr(stream)))

    def step(self, lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, auto_lambda=None):
        """One Adam step (App. D.1: 100 steps at learning rate 1e-2); the first step (at
        the starting point) sets lambda by Eq. 10 unless ``auto_lambda`` is False (then
        ``self.lambdas`` is used as set)."""
        self.t += 1
        auto = (self.t == 1) if auto_lambda is None else bool(auto_lambda)
        _check("kq_calib_step",
               lib().kq_calib_step(_p(self.W), self.M, self.d, self.o, _p(self.theta), _p(self.m), _p(self.v),
                                   self.t, float(lr), float(beta1), float(beta2), float(eps), _p(self.lambdas),
                                   int(auto), _p(self.losses), _p(self.grad), ctypes.c_void_p(self._ws_ptr),
                                   self.ws.numel() - 256, _stream_ptr(self.stream)))
        return self.losses

    def factors(self):
        """The current 2x2 factors, fp32 [d/32][5][2][2] (Eq. 6), for the fused quantizer."""
        return factors_from_lu(self.theta.double().cpu().numpy())


def calib_step_noalloc(A, W, theta, adam_m, adam_v, t, lambdas, losses, grad=None, lr=1e-2, beta1=0.9,
                       beta2=0.999, eps=1e-8, auto_lambda=False, stream=None):
    """One calibration step (kq_calib_init + kq_calib_step) on the library's own
    device workspace (kq_calib_step_noalloc): nothing is allocated. theta, adam_m,
    adam_v, lambdas and losses are updated in place, as by Calibration.step."""
    torch = _torch()
    _dev(A, "A", (torch.bfloat16, torch.int16, torch.uint16))
    _dev(W, "W", (torch.float32,))
    M, d = A.shape
    o = W.shape[0]
    for name, x in (("theta", theta), ("adam_m", adam_m), ("adam_v", adam_v), ("lambdas", lambdas),
                    ("losses", losses)):
        _dev(x, name, (torch.float32,))
    _check("kq_calib_step_noalloc",
           lib().kq_calib_step_noalloc(_p(A), _p(W), M, d, o, _p(theta), _p(adam_m), _p(adam_v), int(t), float(lr),
                                       float(beta1), float(beta2), float(eps), _p(lambdas), int(bool(auto_lambda)),
                                       _p(losses), _p(grad) if grad is not None else None, _stream_ptr(stream)))
    return losses


# ---------------------------------------------------------------------------
# The layer around the W4A4 product: norm in front, epilogue behind, gradients
# ---------------------------------------------------------------------------
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}  # kq_act


def _activation(t, name):
    """(bf16?, device index) of the bf16 or fp32 GPU tensor t."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype is torch.bfloat16:
        return True, t.get_device()
    if t.dtype is torch.float32:
        return False, t.get_device()
    raise TypeError("%s has dtype %s, expected torch.bfloat16 or torch.float32" % (name, t.dtype))


def _elsewhere(index, stream):
    """The context a call on device ``index`` has to run in when it was given a stream or that is
    not the current device (its allocations then belong to that stream too), else None."""
    torch = _torch()
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("the stream is on %s, the tensors on device %d" % (stream.device, index))
        return torch.cuda.stream(stream)
    if index != torch.cuda.current_device():
        return torch.cuda.device(index)
    return None


def _current_stream(index):
    """The current stream of device ``index`` (the current device) as a number. torch.cuda's own
    stream object costs 2.7 us to make, a third of a small call."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream().cuda_stream


def _matrix(t, name, dtype, index, rows=None, cols=None):
    """t's row stride: t must be a [rows][cols] tensor of dtype on device ``index`` with unit column
    stride. A single row's stride does not matter."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected device %d" % (name, t.device, index))
    shape = t.shape
    if len(shape) != 2 or (rows is not None and (shape[0] != rows or shape[1] != cols)):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(shape),
                                                            "[rows][columns]" if rows is None else (rows, cols)))
    stride = t.stride()
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError("%s must have unit column stride" % name)
    return stride[0] if shape[0] > 1 else shape[1]


def _vector(t, name, d, index):
    """Pointer of the fp32 vector t of length d (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not _torch().float32:
        raise TypeError("%s has dtype %s, expected torch.float32" % (name, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected device %d" % (name, t.device, index))
    if t.numel() != d or not t.is_contiguous():
        raise ValueError("%s must be a contiguous fp32 vector of length %d" % (name, d))
    return t.data_ptr()


def _bytes(t, name, rows, cols, index):
    """Pointer of the contiguous uint8 tensor t of rows * cols bytes on device ``index``."""
    torch = _torch()
    if t.dtype is not torch.uint8 or t.get_device() != index:
        raise TypeError("%s must be a uint8 tensor on device %d" % (name, index))
    if t.numel() != rows * cols or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d x %d bytes" % (name, rows, cols))
    return t.data_ptr()


def _packed_scales(t, name, rows, k, index, packed):
    if not packed and tuple(t.shape) != (rows, k // 32):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, k // 32)))
    return _bytes(t, name, rows, k // 32, index)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, rows, cols):
    n = ctypes.c_int64(0)
    _check(name, getattr(lib(), name)(rows, cols, ctypes.byref(n)))
    return n.value


def _workspace(name, rows, cols, workspace, like):
    """(tensor, its bytes) for a call that sums over rows: the caller's, or one of this call's own on
    the device of ``like`` (None where it needs none)."""
    n = _workspace_bytes(name, rows, cols)
    if workspace is None:
        return (like.new_empty(n, dtype=_torch().uint8) if n else None), n
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % like.device)
    return workspace, workspace.numel() * workspace.element_size()


def layernorm(x, weight=None, bias=None, eps=1e-5, out=None, stats=False, mean=None, rstd=None, stream=None):
    """Layer norm of the rows of x (bf16 or fp32 [m][d]): (x - mean) rstd weight + bias, in x's type.

    weight, bias: fp32 [d] or None (1 and 0). ``stats=True`` (or mean, rstd: fp32 [m] to write
    into) returns (y, mean, rstd), what layernorm_backward takes.
    """
    torch = _torch()
    bf16, index = _activation(x, "x")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return layernorm(x, weight, bias, eps, out, stats, mean, rstd)
    ldx = _matrix(x, "x", x.dtype, index)
    m, d = x.shape
    if out is None:
        out, ldy = x.new_empty((m, d)), d
    else:
        ldy = _matrix(out, "out", x.dtype, index, m, d)
    stats = stats or mean is not None or rstd is not None
    if stats:
        if mean is None:
            mean = x.new_empty(m, dtype=torch.float32)
        if rstd is None:
            rstd = x.new_empty(m, dtype=torch.float32)
    _check("kq_layernorm",
           lib().kq_layernorm(x.data_ptr(), int(bf16), m, d, ldx, _vector(weight, "weight", d, index),
                              _vector(bias, "bias", d, index), eps, out.data_ptr(), ldy,
                              _vector(mean, "mean", m, index), _vector(rstd, "rstd", m, index),
                              _current_stream(index)))
    return (out, mean, rstd) if stats else out


def layernorm_backward(dy, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, params=True,
                       workspace=None, stream=None):
    """Gradients of layernorm for its output's gradient dy (x's type and shape): (dx, dweight, dbias).

    mean, rstd: fp32 [m] as layernorm returned them. ``params=False`` computes dx alone (and
    returns None for the others). workspace: at least kq_layernorm_backward_workspace_bytes
    bytes, or None (allocated for this call).
    """
    torch = _torch()
    bf16, index = _activation(x, "x")
    _activation(dy, "dy")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return layernorm_backward(dy, x, mean, rstd, weight, dx, dweight, dbias, params, workspace)
    ldx = _matrix(x, "x", x.dtype, index)
    m, d = x.shape
    lddy = _matrix(dy, "dy", x.dtype, index, m, d)
    if dx is None:
        dx, lddx = x.new_empty((m, d)), d
    else:
        lddx = _matrix(dx, "dx", x.dtype, index, m, d)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are required")
    ws, ws_bytes = None, 0
    if params:
        if dweight is None:
            dweight = x.new_empty(d, dtype=torch.float32)
        if dbias is None:
            dbias = x.new_empty(d, dtype=torch.float32)
        ws, ws_bytes = _workspace("kq_layernorm_backward_workspace_bytes", m, d, workspace, x)
    elif dweight is not None or dbias is not None:
        raise ValueError("params=False computes neither dweight nor dbias")
    _check("kq_layernorm_backward",
           lib().kq_layernorm_backward(dy.data_ptr(), lddy, x.data_ptr(), ldx, int(bf16), m, d,
                                       _vector(weight, "weight", d, index), _vector(mean, "mean", m, index),
                                       _vector(rstd, "rstd", m, index), dx.data_ptr(), lddx,
                                       _vector(dweight, "dweight", d, index), _vector(dbias, "dbias", d, index),
                                       ws.data_ptr() if ws is not None else None, ws_bytes,
                                       _current_stream(index)))
    return dx, dweight, dbias


def layernorm_quantize_mxfp4(x, weight=None, bias=None, factors=None, eps=1e-5, packed=False, codes=None,
                             scales=None, y_debug=None, stats=False, mean=None, rstd=None, stream=None):
    """Layer norm, Kronecker transform (factors fp32 [d/32][5][2][2]; None: T = I) and MXFP4 in one
    pass over x (bf16 or fp32 [m][d]): codes [m][d/2] and scales [m][d/32], or with ``packed``
    in the layout of pack_mxfp4_scales ([d/256][m][8]). No bf16 rounding in between.

    ``y_debug``: optional fp32 [m][d] tensor that receives the transformed norm (check mode).
    ``stats=True`` (or mean, rstd given) returns (codes, scales, mean, rstd).
    """
    torch = _torch()
    bf16, index = _activation(x, "x")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return layernorm_quantize_mxfp4(x, weight, bias, factors, eps, packed, codes, scales, y_debug, stats,
                                            mean, rstd)
    ldx = _matrix(x, "x", x.dtype, index)
    m, d = x.shape
    if codes is None:
        codes = x.new_empty((m, d // 2), dtype=torch.uint8)
    elif tuple(codes.shape) != (m, d // 2):
        raise ValueError("codes has shape %s, expected %s" % (tuple(codes.shape), (m, d // 2)))
    cp = _bytes(codes, "codes", m, d // 2, index)
    if scales is None:
        scales = x.new_empty((d // 256, m, 8) if packed and d % 256 == 0 else (m, d // 32), dtype=torch.uint8)
    sp = _packed_scales(scales, "scales", m, d, index, packed)
    yp = None
    if y_debug is not None:
        if tuple(y_debug.shape) != (m, d):
            raise ValueError("y_debug has shape %s, expected %s" % (tuple(y_debug.shape), (m, d)))
        yp = _vector(y_debug, "y_debug", m * d, index)
    stats = stats or mean is not None or rstd is not None
    if stats:
        if mean is None:
            mean = x.new_empty(m, dtype=torch.float32)
        if rstd is None:
            rstd = x.new_empty(m, dtype=torch.float32)
    _check("kq_layernorm_quantize_mxfp4",
           lib().kq_layernorm_quantize_mxfp4(x.data_ptr(), int(bf16), m, d, ldx, _vector(weight, "weight", d, index),
                                             _vector(bias, "bias", d, index), eps,
                                             _vector(factors, "factors", (d // 32) * 20, index), cp, sp,
                                             1 if packed else 0, yp, _vector(mean, "mean", m, index),
                                             _vector(rstd, "rstd", m, index), _current_stream(index)))
    return (codes, scales, mean, rstd) if stats else (codes, scales)


def mxfp4_linear(codes_a, scales_a, codes_w, scales_w, bias=None, act="none", residual=None, out=None, pre=None,
                 bf16=True, packed=False, want_pre=False, stream=None):
    """act(deq(A) deq(W)^T + bias) + residual from MXFP4 operands, bf16 (or fp32) [m][n].

    Operands as mxfp4_gemm (scales [rows][k/32]; any k % 32 == 0) or, with ``packed``, as
    mxfp4_gemm_packed (k % 256 == 0). bias: fp32 [n]; act: one of ACTS; residual, out, pre: [m][n]
    of the output's type (residual may be out itself). ``want_pre=True`` (or pre given) also returns the values in front of
    the activation, (out, pre), what mxfp4_linear_backward takes.
    """
    torch = _torch()
    if not isinstance(codes_a, torch.Tensor) or not codes_a.is_cuda or codes_a.dtype is not torch.uint8:
        raise TypeError("codes_a must be a uint8 CUDA (HIP) tensor")
    index = codes_a.get_device()
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return mxfp4_linear(codes_a, scales_a, codes_w, scales_w, bias, act, residual, out, pre, bf16, packed,
                                want_pre)
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(ACTS))
    sa, sw = codes_a.shape, codes_w.shape
    if len(sa) != 2 or len(sw) != 2 or sa[1] != sw[1]:
        raise ValueError("codes_a must be [m][k/2] and codes_w [n][k/2], got %s and %s" % (tuple(sa), tuple(sw)))
    m, kb = sa
    n, k = sw[0], 2 * kb
    dtype = torch.bfloat16 if bf16 else torch.float32
    rp = zp = None
    ldr = ldz = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", dtype, index, m, n)
        rp = residual.data_ptr()
    if out is None:
        out, ldo = codes_a.new_empty((m, n), dtype=dtype), n
    else:
        ldo = _matrix(out, "out", dtype, index, m, n)
    if pre is not None:
        ldz = _matrix(pre, "pre", dtype, index, m, n)
        zp = pre.data_ptr()
    elif want_pre:
        pre, ldz = codes_a.new_empty((m, n), dtype=dtype), n
        zp = pre.data_ptr()
    _check("kq_mxfp4_linear",
           lib().kq_mxfp4_linear(_bytes(codes_a, "codes_a", m, kb, index),
                                 _packed_scales(scales_a, "scales_a", m, k, index, packed),
                                 _bytes(codes_w, "codes_w", n, kb, index),
                                 _packed_scales(scales_w, "scales_w", n, k, index, packed), 1 if packed else 0, m, n,
                                 k, _vector(bias, "bias", n, index), ACTS[act], 1 if bf16 else 0, rp, ldr,
                                 out.data_ptr(), ldo, zp, ldz, _current_stream(index)))
    return out if pre is None else (out, pre)


def mxfp4_linear_backward(dout, z=None, act="none", dz=None, dbias=None, workspace=None, stream=None):
    """Gradients of mxfp4_linear's epilogue for its output's gradient dout (bf16 or fp32 [m][n]):
    (dz, dbias) with dz = dout act'(z) and dbias its column sums (fp32 [n]).

    z: the values in front of the activation (mxfp4_linear's pre), may be None with act "none". The
    residual's gradient is dout; the operands' are dz deq(W) and dz^T deq(A).
    """
    torch = _torch()
    bf16, index = _activation(dout, "dout")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return mxfp4_linear_backward(dout, z, act, dz, dbias, workspace)
    dtype = dout.dtype
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(ACTS))
    lddo = _matrix(dout, "dout", dtype, index)
    m, n = dout.shape
    ldz = 0
    if z is not None:
        ldz = _matrix(z, "z", dtype, index, m, n)
    elif act != "none":
        raise ValueError("z is required with act %r" % act)
    if dz is None:
        dz, lddz = dout.new_empty((m, n)), n
    else:
        lddz = _matrix(dz, "dz", dtype, index, m, n)
    if dbias is None:
        dbias = dout.new_empty(n, dtype=torch.float32)
    ws, ws_bytes = _workspace("kq_mxfp4_linear_backward_workspace_bytes", m, n, workspace, dout)
    _check("kq_mxfp4_linear_backward",
           lib().kq_mxfp4_linear_backward(dout.data_ptr(), lddo, None if z is None else z.data_ptr(), ldz, int(bf16),
                                          m, n, ACTS[act], dz.data_ptr(), lddz, _vector(dbias, "dbias", n, index),
                                          ws.data_ptr() if ws is not None else None, ws_bytes,
                                          _current_stream(index)))
    return dz, dbias


def _sums(t, name, d, index, like):
    """(fp32 vector of length d, its pointer): t, or one of this call's own on the device of ``like``."""
    if t is None:
        t = like.new_empty(d, dtype=_torch().float32)
        return t, t.data_ptr()
    return t, _vector(t, name, d, index)


def mxfp4_gated_linear(codes_a, scales_a, codes_g, scales_g, codes_u, scales_u, bias_g=None, bias_u=None, act="silu",
                       out=None, g=None, u=None, bf16=True, packed=False, want_pre=False, stream=None):
    """act(deq(A) deq(Wg)^T + bias_g) * (deq(A) deq(Wu)^T + bias_u) from MXFP4 operands, bf16 (or fp32) [m][n]: both
    projections of a gated feed-forward block in one kernel.

    Operands, ``packed`` and act as mxfp4_linear; bias_g, bias_u: fp32 [n]; out, g, u: [m][n] of the output's
    type. ``want_pre=True`` (or g or u given) also returns the two products, (out, g, u), what
    mxfp4_gated_linear_backward takes.
    """
    torch = _torch()
    if not isinstance(codes_a, torch.Tensor) or not codes_a.is_cuda or codes_a.dtype is not torch.uint8:
        raise TypeError("codes_a must be a uint8 CUDA (HIP) tensor")
    index = codes_a.get_device()
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return mxfp4_gated_linear(codes_a, scales_a, codes_g, scales_g, codes_u, scales_u, bias_g, bias_u, act, out,
                                      g, u, bf16, packed, want_pre)
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(ACTS))
    sa, sg, su = codes_a.shape, codes_g.shape, codes_u.shape
    if len(sa) != 2 or len(sg) != 2 or sg != su or sa[1] != sg[1]:
        raise ValueError("codes_a must be [m][k/2] and codes_g, codes_u [n][k/2], got %s, %s and %s" % (
            tuple(sa), tuple(sg), tuple(su)))
    m, kb = sa
    n, k = sg[0], 2 * kb
    dtype = torch.bfloat16 if bf16 else torch.float32
    if out is None:
        out, ldo = codes_a.new_empty(m, n, dtype=dtype), n
    else:
        ldo = _matrix(out, "out", dtype, index, m, n)
    gp = up = None
    ldg = ldu = 0
    want_pre = want_pre or g is not None or u is not None
    if want_pre:
        if g is None:
            g = codes_a.new_empty(m, n, dtype=dtype)
        if u is None:
            u = codes_a.new_empty(m, n, dtype=dtype)
        ldg, ldu = _matrix(g, "g", dtype, index, m, n), _matrix(u, "u", dtype, index, m, n)
        gp, up = g.data_ptr(), u.data_ptr()
    _check("kq_mxfp4_gated_linear",
           lib().kq_mxfp4_gated_linear(_bytes(codes_a, "codes_a", m, kb, index),
                                       _packed_scales(scales_a, "scales_a", m, k, index, packed),
                                       _bytes(codes_g, "codes_g", n, kb, index),
                                       _packed_scales(scales_g, "scales_g", n, k, index, packed),
                                       _bytes(codes_u, "codes_u", n, kb, index),
                                       _packed_scales(scales_u, "scales_u", n, k, index, packed), 1 if packed else 0, m,
                                       n, k, _vector(bias_g, "bias_g", n, index), _vector(bias_u, "bias_u", n, index),
                                       ACTS[act], 1 if bf16 else 0, out.data_ptr(), ldo, gp, ldg, up, ldu,
                                       _current_stream(index)))
    return (out, g, u) if want_pre else out


def mxfp4_gated_linear_backward(dout, g, u, act="silu", dg=None, du=None, dbias_g=None, dbias_u=None, biases=True,
                                workspace=None, stream=None):
    """Gradients of mxfp4_gated_linear's epilogue for its output's gradient dout (bf16 or fp32 [m][n]):
    (dg, du, dbias_g, dbias_u) with dg = dout u act'(g), du = dout act(g) and the biases' their column sums (fp32 [n]).

    g, u: the two products (mxfp4_gated_linear's). ``biases=False``: None for the sums. dg and du may be halves of
    one [m][2 n] tensor. The operands' gradients are dg deq(Wg) + du deq(Wu), dg^T deq(A) and du^T deq(A).
    """
    bf16, index = _activation(dout, "dout")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return mxfp4_gated_linear_backward(dout, g, u, act, dg, du, dbias_g, dbias_u, biases, workspace)
    dtype = dout.dtype
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(ACTS))
    lddo = _matrix(dout, "dout", dtype, index)
    m, n = dout.shape
    ldg, ldu = _matrix(g, "g", dtype, index, m, n), _matrix(u, "u", dtype, index, m, n)
    if dg is None:
        dg, lddg = dout.new_empty(m, n), n
    else:
        lddg = _matrix(dg, "dg", dtype, index, m, n)
    if du is None:
        du, lddu = dout.new_empty(m, n), n
    else:
        lddu = _matrix(du, "du", dtype, index, m, n)
    ws, ws_bytes = None, 0
    gp = up = None
    if biases:
        dbias_g, gp = _sums(dbias_g, "dbias_g", n, index, dout)
        dbias_u, up = _sums(dbias_u, "dbias_u", n, index, dout)
        ws, ws_bytes = _workspace("kq_mxfp4_gated_linear_backward_workspace_bytes", m, n, workspace, dout)
    elif dbias_g is not None or dbias_u is not None:
        raise ValueError("biases=False computes neither dbias_g nor dbias_u")
    _check("kq_mxfp4_gated_linear_backward",
           lib().kq_mxfp4_gated_linear_backward(dout.data_ptr(), lddo, g.data_ptr(), ldg, u.data_ptr(), ldu, int(bf16), m,
                                                n, ACTS[act], dg.data_ptr(), lddg, du.data_ptr(), lddu,
                                                gp, up,
                                                ws.data_ptr() if ws is not None else None, ws_bytes,
                                                _current_stream(index)))
    return dg, du, dbias_g, dbias_u


# ---------------------------------------------------------------------------
# Queries, keys and values: norm and rotation of heads, the MXFP4 cache
# ---------------------------------------------------------------------------
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}  # kq_rope_scaling


class _Rope(ctypes.Structure):  # kq_rope, for calls of lib() itself
    _fields_ = [("positions", ctypes.c_void_p), ("freq", ctypes.c_void_p), ("rot", ctypes.c_int64),
                ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float), ("axes", ctypes.c_int),
                ("axis_pairs", ctypes.c_int64 * 4)]


_ROPE = struct.Struct("@PPqifi4xqqqq")  # its bytes, a third of the time of filling in a _Rope


def rope_frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """Host helper: the frequencies (radians per position, float64 [rot / 2]) of a rotation of ``rot``
    channels, base^(-2 i / rot), scaled for contexts longer than those of training (kq_rope_frequencies): "linear"
    divides them by factor, "base" stretches the base so that the lowest is, "parts" divides those of
    fewer than ``low`` turns in ``original`` positions, keeps those of more than ``high`` and blends between."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(ROPE_SCALINGS))
    out = np.empty(max(0, rot // 2), dtype=np.float64)
    _check("kq_rope_frequencies",
           lib().kq_rope_frequencies(rot, base, ROPE_SCALINGS[scaling], factor, original, low, high,
                                     ctypes.c_void_p(out.ctypes.data)))
    return out


def _rope(positions, freq, m, index, interleaved, amplitude, axis_pairs):
    """kq_rope of the rotation's arguments on device ``index``, as bytes (freq None: NULL)."""
    if freq is None:
        return None
    torch = _torch()
    if not isinstance(freq, torch.Tensor) or freq.dtype is not torch.float64 or freq.dim() != 1 or not freq.is_contiguous():
        raise TypeError("freq must be a contiguous float64 vector")
    if positions is None or positions.dtype is not torch.int64 or not positions.is_contiguous():
        raise TypeError("positions must be a contiguous int64 tensor")
    if freq.get_device() != index or positions.get_device() != index:
        raise ValueError("positions and freq must be on device %d" % index)
    shape = positions.shape
    axes = 1 if len(shape) == 1 else shape[1] if len(shape) == 2 else 0
    if len(shape) == 0 or shape[0] != m or not 1 <= axes <= 4:
        raise ValueError("positions has shape %s, expected [%d] or [%d][1 to 4 axes]" % (tuple(shape), m, m))
    n = freq.shape[0]
    pairs = tuple(axis_pairs) if axis_pairs is not None else (n,)
    if len(pairs) != axes:
        raise ValueError("axis_pairs must name the pairs of each of the %d axes" % axes)
    return _ROPE.pack(positions.data_ptr(), freq.data_ptr(), 2 * n, 1 if interleaved else 0, amplitude, axes,
                      *pairs, *(0,) * (4 - axes))


def _heads(t, name, dtype, index, shape=None):
    """t's token and head strides: a [tokens][heads][channels] tensor of dtype on device ``index`` with
    unit channel stride. The stride of a single token or head does not matter."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected device %d" % (name, t.device, index))
    got = t.shape
    if len(got) != 3 or (shape is not None and got != shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(got), "[tokens][heads][channels]"
                                                            if shape is None else tuple(shape)))
    ld, hs, c = t.stride()
    if c != 1 and got[2] > 1:
        raise ValueError("%s must have unit channel stride" % name)
    return ld if got[0] > 1 else got[1] * got[2], hs if got[1] > 1 else got[2]


def headnorm_rope(x, positions=None, freq=None, weight_q=None, weight_k=None, q_heads=None, norm=True, eps=1e-6,
                  interleaved=False, amplitude=1.0, axis_pairs=None, out=None, stream=None):
    """The norm of each head of x (bf16 or fp32 [m][heads][d], a view of a product's output say) and the rotation
    of its position, in x's type: x w / sqrt(mean(x^2) + eps), then the first 2 len(freq) channels turned
    by positions freq.

    weight_q: fp32 [d], of the first ``q_heads`` heads (None: all); weight_k: of the others; None: 1.
    ``norm=False``: the rotation alone. positions: int64 [m] or [m][axes]; freq: float64, one per
    pair (rope_frequencies; None: no rotation); axis_pairs: how many pairs turn with each axis. Pairs are
    (i, i + len(freq)), or (2 i, 2 i + 1) with ``interleaved``; amplitude multiplies the rotated
    channels. out: [m][heads][d] of any strides (x itself: in place).
    """
    bf16, index = _activation(x, "x")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return headnorm_rope(x, positions, freq, weight_q, weight_k, q_heads, norm, eps, interleaved, amplitude,
                                 axis_pairs, out)
    ldx, hsx = _heads(x, "x", x.dtype, index)
    m, heads, d = x.shape
    if out is None:
        out, ldy, hsy = x.new_empty(m, heads, d), heads * d, d
    else:
        ldy, hsy = _heads(out, "out", x.dtype, index, x.shape)
    _check("kq_headnorm_rope",
           lib().kq_headnorm_rope(x.data_ptr(), int(bf16), m, heads, d, ldx, hsx, 1 if norm else 0,
                                  _vector(weight_q, "weight_q", d, index), _vector(weight_k, "weight_k", d, index),
                                  heads if q_heads is None else q_heads, eps,
                                  _rope(positions, freq, m, index, interleaved, amplitude, axis_pairs),
                                  out.data_ptr(), ldy, hsy, _current_stream(index)))
    return out


def headnorm_rope_backward(dy, x=None, positions=None, freq=None, weight_q=None, weight_k=None, q_heads=None,
                           norm=True, eps=1e-6, interleaved=False, amplitude=1.0, axis_pairs=None, dx=None,
                           dweight_q=None, dweight_k=None, params=True, workspace=None, stream=None):
    """Gradients of headnorm_rope for its output's gradient dy (x's type and shape): (dx, dweight_q, dweight_k).

    ``params=False`` (or ``norm=False``, where x is not needed) computes dx alone, with None for the
    others. workspace: at least kq_headnorm_rope_backward_workspace_bytes bytes, or None
    (allocated for this call). The rest as headnorm_rope.
    """
    bf16, index = _activation(dy, "dy")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return headnorm_rope_backward(dy, x, positions, freq, weight_q, weight_k, q_heads, norm, eps, interleaved,
                                          amplitude, axis_pairs, dx, dweight_q, dweight_k, params, workspace)
    lddy, hsdy = _heads(dy, "dy", dy.dtype, index)
    m, heads, d = dy.shape
    ldx = hsx = 0
    if norm:
        if x is None:
            raise ValueError("x is required with norm=True")
        ldx, hsx = _heads(x, "x", dy.dtype, index, dy.shape)
    if dx is None:
        dx, lddx, hsdx = dy.new_empty(m, heads, d), heads * d, d
    else:
        lddx, hsdx = _heads(dx, "dx", dy.dtype, index, dy.shape)
    ws, ws_bytes = None, 0
    qp = kp = None
    if params and norm:
        dweight_q, qp = _sums(dweight_q, "dweight_q", d, index, dy)
        dweight_k, kp = _sums(dweight_k, "dweight_k", d, index, dy)
        ws, ws_bytes = _workspace("kq_headnorm_rope_backward_workspace_bytes", m, d, workspace, dy)
    elif dweight_q is not None or dweight_k is not None:
        raise ValueError("params=False and norm=False compute no dweight")
    _check("kq_headnorm_rope_backward",
           lib().kq_headnorm_rope_backward(dy.data_ptr(), lddy, hsdy, x.data_ptr() if norm else None, ldx, hsx,
                                           int(bf16), m, heads, d, 1 if norm else 0,
                                           _vector(weight_q, "weight_q", d, index),
                                           _vector(weight_k, "weight_k", d, index),
                                           heads if q_heads is None else q_heads, eps,
                                           _rope(positions, freq, m, index, interleaved, amplitude, axis_pairs),
                                           dx.data_ptr(), lddx, hsdx, qp, kp,
                                           ws.data_ptr() if ws is not None else None, ws_bytes,
                                           _current_stream(index)))
    return dx, dweight_q, dweight_k


def _slots(t, index):
    """Pointer of the int64 slot list t on device ``index``."""
    if not isinstance(t, _torch().Tensor) or t.dtype is not _torch().int64 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError("slots must be a contiguous int64 vector")
    if t.get_device() != index:
        raise ValueError("slots is on %s, expected device %d" % (t.device, index))
    return t.data_ptr()


def _cache(codes, scales, name, heads, d, index, slots=None):
    """(slots, codes pointer, scales pointer) of one half of a cache."""
    if codes is None or scales is None:
        raise ValueError("codes%s and scales%s are required" % (name, name))
    n = codes.shape[0]
    if tuple(codes.shape) != (n, heads, d // 2) or tuple(scales.shape) != (n, heads, d // 32) or slots not in (None, n):
        raise ValueError("codes%s and scales%s have shapes %s and %s, expected [slots][%d][%d] and [slots][%d][%d]" % (
            name, name, tuple(codes.shape), tuple(scales.shape), heads, d // 2, heads, d // 32))
    return (n, _bytes(codes, "codes" + name, n * heads, d // 2, index),
            _bytes(scales, "scales" + name, n * heads, d // 32, index))


def cache_write_mxfp4(slots, k=None, codes_k=None, scales_k=None, v=None, codes_v=None, scales_v=None,
                      norm=False, weight=None, eps=1e-6, positions=None, freq=None, interleaved=False, amplitude=1.0,
                      axis_pairs=None, stream=None):
    """Quantizes keys and values (bf16 or fp32 [m][heads][d]; either may be None) into their cache of MXFP4: codes
    uint8 [slots][heads][d/2] and scales uint8 [slots][heads][d/32]. Token i goes to slot slots[i] (int64 [m]);
    one that is negative or past the cache is left out, and two tokens must not share one. Keys are normed (``norm``, with weight) and rotated
    first, as by headnorm_rope, without a rounding in between; values go in as they are.
    """
    one = k if k is not None else v
    if one is None:
        raise ValueError("keys or values are required")
    bf16, index = _activation(one, "k" if k is not None else "v")
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return cache_write_mxfp4(slots, k, codes_k, scales_k, v, codes_v, scales_v, norm, weight, eps, positions,
                                     freq, interleaved, amplitude, axis_pairs)
    m, _, d = one.shape if one.dim() == 3 else (0, 0, 0)
    n, parts = None, []
    for t, codes, scales, name in ((k, codes_k, scales_k, "_k"), (v, codes_v, scales_v, "_v")):
        if t is None:
            parts.append((None, 0, 0, 0, None, None))
            continue
        ld, hs = _heads(t, name[1:], one.dtype, index)
        heads = t.shape[1]
        if t.shape[0] != m or t.shape[2] != d:
            raise ValueError("k and v must have the same tokens and channels, got %s and %s" % (tuple(k.shape), tuple(v.shape)))
        n, cp, sp = _cache(codes, scales, name, heads, d, index, n)
        parts.append((t.data_ptr(), ld, hs, heads, cp, sp))
    (kp, ldk, hsk, kh, ckp, skp), (vp, ldv, hsv, vh, cvp, svp) = parts
    sp = _slots(slots, index)
    if slots.numel() != m:
        raise ValueError("slots has %d entries, expected %d" % (slots.numel(), m))
    _check("kq_cache_write_mxfp4",
           lib().kq_cache_write_mxfp4(kp, ldk, hsk, kh, vp, ldv, hsv, vh, int(bf16), m, d, 1 if norm else 0,
                                      _vector(weight, "weight", d, index), eps,
                                      _rope(positions, freq, m, index, interleaved, amplitude, axis_pairs),
                                      sp, n, ckp, skp, cvp, svp, _current_stream(index)))


def cache_read_mxfp4(slots, codes, scales, bf16=True, out=None, stream=None):
    """The rows slots[i] (int64 [m]) of a cache of keys or of values (codes uint8 [slots][heads][d/2], scales uint8
    [slots][heads][d/32]) decoded, bf16 (or fp32) [m][heads][d], exactly. A slot that is negative or past the
    cache reads as zeros. out: [m][heads][d] of any strides.
    """
    torch = _torch()
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dim() != 3:
        raise TypeError("codes must be a CUDA (HIP) tensor [slots][heads][d/2]")
    index = codes.get_device()
    here = _elsewhere(index, stream)
    if here is not None:
        with here:
            return cache_read_mxfp4(slots, codes, scales, bf16, out)
    heads, d = codes.shape[1], 2 * codes.shape[2]
    n, cp, sp = _cache(codes, scales, "", heads, d, index)
    dtype = torch.bfloat16 if bf16 else torch.float32
    slots_p, m = _slots(slots, index), slots.numel()
    if out is None:
        out, ldy, hsy = codes.new_empty(m, heads, d, dtype=dtype), heads * d, d
    else:
        ldy, hsy = _heads(out, "out", dtype, index, (m, heads, d))
    _check("kq_cache_read_mxfp4",
           lib().kq_cache_read_mxfp4(slots_p, m, cp, sp, n, heads, d, 1 if bf16 else 0, out.data_ptr(),
                                     ldy, hsy, _current_stream(index)))
    return out


def factors_from_lu(abc):
    """Host helper: (a, b, c) per factor, fp64 [nblk][5][3] -> fp32 [nblk][5][2][2] (Eq. 6)."""
    abc = np.ascontiguousarray(abc, dtype=np.float64)
    nblk = abc.shape[0]
    out = np.empty((nblk, 5, 2, 2), dtype=np.float32)
    _check("kq_factors_from_lu",
           lib().kq_factors_from_lu(ctypes.c_void_p(abc.ctypes.data), nblk,
                                    ctypes.c_void_p(out.ctypes.data)))
    return out
