"""Microscaled 4-bit floating point over torch device tensors: quantise,
dequantise and multiply (include/qamw.h states the format).

A quantised matrix is the pair (codes [N][qamw_mxfp4_row_bytes(d)],
scales [N][qamw_mxfp4_scale_bytes(d)]), both uint8.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .codec import _ODT, _dev, _rows, _stream, _temporary

__all__ = [
    "qamw_mxfp4_dequantize",
    "qamw_mxfp4_matmul",
    "qamw_mxfp4_matmul_workspace_bytes",
    "qamw_mxfp4_quantize",
    "qamw_mxfp4_row_bytes",
    "qamw_mxfp4_scale_bytes",
]


def qamw_mxfp4_row_bytes(d: int) -> int:
    return int(_lib.load().qamw_mxfp4_row_bytes(d))


def qamw_mxfp4_scale_bytes(d: int) -> int:
    return int(_lib.load().qamw_mxfp4_scale_bytes(d))


def qamw_mxfp4_matmul_workspace_bytes(T: int, N: int, d: int) -> int:
    return int(_lib.load().qamw_mxfp4_matmul_workspace_bytes(T, N, d))


def _pitch(W: torch.Tensor, name: str):
    """Rows, columns and a leading dimension of at least the columns (an empty or one-row matrix has none of its own)."""
    n, d, ld = _rows(W, name)
    return n, d, max(ld, d) if n <= 1 else ld


def _quantised(codes: torch.Tensor, scales: torch.Tensor, d: int) -> int:
    _dev(codes, "codes")
    _dev(scales, "scales")
    lib = _lib.load()
    rb, sb = int(lib.qamw_mxfp4_row_bytes(d)), int(lib.qamw_mxfp4_scale_bytes(d))
    if rb < 0:
        raise ValueError(f"unsupported d={d}")
    N = codes.shape[0] if codes.dim() == 2 else -1
    for t, name, width in ((codes, "codes", rb), (scales, "scales", sb)):
        if t.dtype != torch.uint8 or tuple(t.shape) != (N, width) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor of {width} columns (d={d}), a row per matrix row")
    return N


def qamw_mxfp4_quantize(W: torch.Tensor, values_dtype=None, codes: Optional[torch.Tensor] = None,
                        scales: Optional[torch.Tensor] = None, values: Optional[torch.Tensor] = None, stream=None):
    """W [N][d] (fp32, bf16 or fp16) -> (codes, scales), or (codes, scales, values) when values_dtype or values is
    given: values [N][d] is what the codes stand for, as qamw_output_error's W_hat."""
    N, d, ldw = _pitch(W, "W")
    if W.dtype not in _ODT:
        raise ValueError("W must be float32, bfloat16 or float16")
    lib = _lib.load()
    rb = int(lib.qamw_mxfp4_row_bytes(d))
    if rb < 0:
        raise ValueError(f"unsupported d={d}")
    if codes is None:
        codes = torch.empty((N, rb), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N, int(lib.qamw_mxfp4_scale_bytes(d))), dtype=torch.uint8, device=W.device)
    if _quantised(codes, scales, d) != N:
        raise ValueError(f"codes and scales must have {N} rows")
    if values is None and values_dtype is not None:
        values = torch.empty((N, d), dtype=values_dtype, device=W.device)
    vptr, vdt, ldv = None, _lib.QAMW_F32, d
    if values is not None:
        n2, d2, ldv = _pitch(values, "values")
        if (n2, d2) != (N, d) or values.dtype not in _ODT or (values_dtype or values.dtype) != values.dtype:
            raise ValueError("values must be N x d of values_dtype: float32, bfloat16 or float16")
        vptr, vdt = values.data_ptr(), _ODT[values.dtype]
    _lib.check("qamw_mxfp4_quantize", lib.qamw_mxfp4_quantize(
        W.data_ptr(), _ODT[W.dtype], N, d, ldw, codes.data_ptr(), scales.data_ptr(), vptr, vdt, ldv, _stream(stream)))
    return (codes, scales) if values is None else (codes, scales, values)


def qamw_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, d: int, out_dtype=torch.float32,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The [N][d] values of a quantised matrix in out_dtype (fp32, bf16 or fp16)."""
    N = _quantised(codes, scales, d)
    if out is None:
        out = torch.empty((N, d), dtype=out_dtype, device=codes.device)
    n2, d2, ldo = _pitch(out, "out")
    if (n2, d2) != (N, d) or out.dtype not in _ODT:
        raise ValueError("out must be N x d of float32, bfloat16 or float16")
    _lib.check("qamw_mxfp4_dequantize", _lib.load().qamw_mxfp4_dequantize(
        codes.data_ptr(), scales.data_ptr(), N, d, out.data_ptr(), _ODT[out.dtype], ldo, _stream(stream)))
    return out


def qamw_mxfp4_matmul(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y [T][N] = X^ W^^T in out_dtype (fp32 or bf16): W^ the quantised matrix, X^ the activations X [T][d] (fp32,
    bf16 or fp16) quantised by the same rule within the call."""
    T, d, ldx = _pitch(X, "X")
    if X.dtype not in _ODT:
        raise ValueError("X must be float32, bfloat16 or float16")
    N = _quantised(codes, scales, d)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=X.device)
    t2, n2, ldy = _pitch(out, "out")
    if (t2, n2) != (T, N) or out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out must be T x N of float32 or bfloat16")
    lib = _lib.load()
    if workspace is None:
        workspace = _temporary(int(lib.qamw_mxfp4_matmul_workspace_bytes(T, N, d)), X.device, stream)
    _dev(workspace, "workspace")
    _lib.check("qamw_mxfp4_matmul", lib.qamw_mxfp4_matmul(
        X.data_ptr(), _ODT[X.dtype], T, d, ldx, codes.data_ptr(), scales.data_ptr(), N, out.data_ptr(),
        _ODT[out.dtype], ldy, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)))
    return out
