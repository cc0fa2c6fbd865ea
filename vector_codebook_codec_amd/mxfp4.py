"""Microscaled 4-bit floating point over torch device tensors: quantise,
dequantise, multiply, and multiply with low-rank adapters of many requests
beside the shared weights (include/qamw.h states the format).

A quantised matrix is the pair (codes [N][qamw_mxfp4_row_bytes(d)],
scales [N][qamw_mxfp4_scale_bytes(d)]), both uint8.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .codec import _ODT, _WDT, _dev, _empty, _matrix, _one_device, _raw_stream, _workspace

__all__ = [
    "qamw_mxfp4_adapter_matmul",
    "qamw_mxfp4_adapter_matmul_workspace_bytes",
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


def _sizes(d: int):
    """Bytes of a row of codes and of a row of scales (the library's qamw_mxfp4_row_bytes and _scale_bytes)."""
    if not 1 <= d <= 1 << 20:
        raise ValueError(f"unsupported d={d}")
    blocks = (d + 31) >> 5
    return blocks << 4, (blocks + 15) & ~15


def _quantised(codes: torch.Tensor, scales: torch.Tensor, d: int) -> int:
    rb, sb = _sizes(d)
    N = codes.shape[0] if codes.dim() == 2 else -1
    for t, name, width in ((codes, "codes", rb), (scales, "scales", sb)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.dtype is not torch.uint8 or t.shape != (N, width) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor of {width} columns (d={d}), a row per matrix row")
    return N


def qamw_mxfp4_quantize(W: torch.Tensor, values_dtype=None, codes: Optional[torch.Tensor] = None,
                        scales: Optional[torch.Tensor] = None, values: Optional[torch.Tensor] = None, stream=None):
    """W [N][d] (fp32, bf16 or fp16) -> (codes, scales), or (codes, scales, values) when values_dtype or values is
    given: values [N][d] is what the codes stand for, as qamw_output_error's W_hat."""
    N, d, ldw = _matrix(W, "W")
    wdt = _ODT.get(W.dtype)
    if wdt is None:
        raise ValueError("W must be float32, bfloat16 or float16")
    rb, sb = _sizes(d)
    if codes is None and scales is None:
        codes = _empty((N, rb), torch.uint8, W.device, stream)
        scales = _empty((N, sb), torch.uint8, W.device, stream)
    else:
        codes = _empty((N, rb), torch.uint8, W.device, stream) if codes is None else codes
        scales = _empty((N, sb), torch.uint8, W.device, stream) if scales is None else scales
        if _quantised(codes, scales, d) != N:
            raise ValueError(f"codes and scales must have {N} rows")
    vptr, vdt, ldv = None, 0, d
    if values is not None or values_dtype is not None:
        if values is None:
            values = _empty((N, d), values_dtype, W.device, stream)
        n2, d2, ldv = _matrix(values, "values")
        vdt = _ODT.get(values.dtype)
        if n2 != N or d2 != d or vdt is None or (values_dtype or values.dtype) != values.dtype:
            raise ValueError("values must be N x d of values_dtype: float32, bfloat16 or float16")
        vptr = values.data_ptr()
    status = _lib.load().qamw_mxfp4_quantize(W.data_ptr(), wdt, N, d, ldw, codes.data_ptr(), scales.data_ptr(), vptr, vdt,
                                             ldv, _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_quantize", status)
    return (codes, scales) if values is None else (codes, scales, values)


def qamw_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, d: int, out_dtype=torch.float32,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The [N][d] values of a quantised matrix in out_dtype (fp32, bf16 or fp16)."""
    N = _quantised(codes, scales, d)
    if out is None:
        out = _empty((N, d), out_dtype, codes.device, stream)
    n2, d2, ldo = _matrix(out, "out")
    odt = _ODT.get(out.dtype)
    if n2 != N or d2 != d or odt is None:
        raise ValueError("out must be N x d of float32, bfloat16 or float16")
    status = _lib.load().qamw_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), N, d, out.data_ptr(), odt, ldo,
                                               _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_dequantize", status)
    return out


def qamw_mxfp4_matmul(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Y [T][N] = X^ W^^T in out_dtype (fp32 or bf16): W^ the quantised matrix, X^ the activations X [T][d] (fp32,
    bf16 or fp16) quantised by the same rule within the call."""
    T, d, ldx = _matrix(X, "X")
    xdt = _ODT.get(X.dtype)
    if xdt is None:
        raise ValueError("X must be float32, bfloat16 or float16")
    N = _quantised(codes, scales, d)
    if out is None:
        out = _empty((T, N), out_dtype, X.device, stream)
    t2, n2, ldy = _matrix(out, "out")
    ydt = _WDT.get(out.dtype)
    if t2 != T or n2 != N or ydt is None:
        raise ValueError("out must be T x N of float32 or bfloat16")
    lib = _lib.load()
    if workspace is None:
        workspace = _workspace(lib.qamw_mxfp4_matmul_workspace_bytes(T, N, d), X.device, stream)
    else:
        _dev(workspace, "workspace")
    status = lib.qamw_mxfp4_matmul(X.data_ptr(), xdt, T, d, ldx, codes.data_ptr(), scales.data_ptr(), N, out.data_ptr(), ydt,
                                   ldy, workspace.data_ptr(), workspace.nbytes, _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_matmul", status)
    return out


def qamw_mxfp4_adapter_matmul_workspace_bytes(T: int, N: int, d: int, rank: int, dtype=torch.bfloat16) -> int:
    return int(_lib.load().qamw_mxfp4_adapter_matmul_workspace_bytes(T, N, d, rank, _WDT[dtype]))


def qamw_mxfp4_adapter_matmul(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                              index: torch.Tensor, factors: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """Y [T][N] = X^ W^^T + factors[i] (X A_i^T) B_i^T with i = index[t] for token t, in out_dtype (fp32 or bf16): the
    product of qamw_mxfp4_matmul with every request's own low-rank adapter.

    X [T][d], A [adapters][rank][d] and B [adapters][N][rank] fp32 or bf16 alike, A and B contiguous; index [T] int32,
    outside [0, adapters) for a token without one; factors [adapters] fp32 (1 if not given).  All lie on the current device."""
    T, d, ldx = _matrix(X, "X")
    xdt = _WDT.get(X.dtype)
    if xdt is None:
        raise ValueError("X must be float32 or bfloat16")
    N = _quantised(codes, scales, d)
    _dev(A, "A")
    _dev(B, "B")
    n, rank = (A.shape[0], A.shape[1]) if A.dim() == 3 else (-1, -1)
    if A.shape != (n, rank, d) or B.shape != (n, N, rank) or A.dtype is not X.dtype or B.dtype is not X.dtype or \
            not A.is_contiguous() or not B.is_contiguous():
        raise ValueError("A must be [adapters][rank][d] and B [adapters][N][rank], contiguous and of X's dtype")
    _dev(index, "index")
    if index.dtype is not torch.int32 or index.shape != (T,) or not index.is_contiguous():
        raise ValueError("index must be a contiguous int32 tensor with an entry per row of X")
    if factors is not None:
        _dev(factors, "factors")
        if factors.dtype is not torch.float32 or factors.shape != (n,) or not factors.is_contiguous():
            raise ValueError("factors must be a contiguous float32 tensor with an entry per adapter")
    if out is None:
        out = _empty((T, N), out_dtype, X.device, stream)
    t2, n2, ldy = _matrix(out, "out")
    ydt = _WDT.get(out.dtype)
    if t2 != T or n2 != N or ydt is None:
        raise ValueError("out must be T x N of float32 or bfloat16")
    lib = _lib.load()
    if workspace is None:
        workspace = _workspace(lib.qamw_mxfp4_adapter_matmul_workspace_bytes(T, N, d, rank, xdt), X.device, stream)
    else:
        _dev(workspace, "workspace")
    _one_device(X, codes=codes, scales=scales, A=A, B=B, index=index, factors=factors, out=out, workspace=workspace)
    status = lib.qamw_mxfp4_adapter_matmul(
        X.data_ptr(), xdt, T, d, ldx, codes.data_ptr(), scales.data_ptr(), N, A.data_ptr(), B.data_ptr(), n, rank,
        index.data_ptr(), None if factors is None else factors.data_ptr(), out.data_ptr(), ydt, ldy, workspace.data_ptr(),
        workspace.nbytes, _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_adapter_matmul", status)
    return out
