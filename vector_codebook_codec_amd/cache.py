"""An attention cache in microscaled 4-bit floating point over torch device
tensors: keys and values quantised as they are written, read back, and
attended to in place (include/qamw.h states the layout).

A cache is the pair (codes [2][pages][heads][page][qamw_mxfp4_cache_row_bytes(d)],
scales [2][pages][heads][page][qamw_mxfp4_cache_scale_bytes(d)]), both uint8,
keys first.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .codec import _ODT, _dev, _empty, _one_device, _raw_stream, _workspace

__all__ = [
    "qamw_mxfp4_cache_attention",
    "qamw_mxfp4_cache_attention_workspace_bytes",
    "qamw_mxfp4_cache_new",
    "qamw_mxfp4_cache_read",
    "qamw_mxfp4_cache_row_bytes",
    "qamw_mxfp4_cache_scale_bytes",
    "qamw_mxfp4_cache_write",
]


def qamw_mxfp4_cache_row_bytes(d: int) -> int:
    return int(_lib.load().qamw_mxfp4_cache_row_bytes(d))


def qamw_mxfp4_cache_scale_bytes(d: int) -> int:
    return int(_lib.load().qamw_mxfp4_cache_scale_bytes(d))


def qamw_mxfp4_cache_attention_workspace_bytes(T: int, sequences: int, max_queries: int, heads: int, q_heads: int, d: int,
                                               tokens: int, q_dtype=torch.bfloat16, out_dtype=torch.bfloat16) -> int:
    """tokens: columns of the page table times the page."""
    return int(_lib.load().qamw_mxfp4_cache_attention_workspace_bytes(T, sequences, max_queries, heads, q_heads, d, tokens,
                                                                      _ODT[q_dtype], _ODT[out_dtype]))


def _sizes(d: int):
    """Bytes of a row of codes and of a row of scales (the library's two size functions)."""
    if not 1 <= d <= 256:
        raise ValueError(f"unsupported head dimension {d}")
    blocks = (d + 31) >> 5
    return blocks << 4, 2 if blocks <= 2 else 4 if blocks <= 4 else 8


def qamw_mxfp4_cache_new(pages: int, heads: int, page: int, d: int, device="cuda"):
    """An empty cache: (codes, scales), every value 0."""
    rb, sb = _sizes(d)
    return (torch.zeros(2, pages, heads, page, rb, dtype=torch.uint8, device=device),
            torch.zeros(2, pages, heads, page, sb, dtype=torch.uint8, device=device))


def _cache(codes: torch.Tensor, scales: torch.Tensor, d: int):
    """(pages, heads, page) of a cache for heads of d elements."""
    rb, sb = _sizes(d)
    if not isinstance(codes, torch.Tensor) or codes.dim() != 5:
        raise ValueError("codes must be a GPU tensor [2][pages][heads][page][row bytes]")
    _, pages, heads, page, _ = codes.shape
    for t, name, width in ((codes, "codes", rb), (scales, "scales", sb)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.dtype is not torch.uint8 or t.shape != (2, pages, heads, page, width) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor [2][pages][heads][page][{width}] (d={d})")
    return pages, heads, page


def _head_rows(t: torch.Tensor, name: str):
    """(dtype code, tokens, heads, d, token stride, head stride) of a tensor with unit stride along the head."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    dt = _ODT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [tokens][heads][d] with unit stride along d")
    T, heads, d = t.shape
    st, sh, _ = t.stride()
    return dt, T, heads, d, st, sh


def _ints(t: torch.Tensor, name: str, dtype, *shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype is not dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}")


def _empty_heads(T: int, heads: int, d: int, dtype, device, stream) -> torch.Tensor:
    return _empty((T, heads * d), dtype, device, stream).view(T, heads, d)


def qamw_mxfp4_cache_write(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                           stream=None) -> None:
    """K and V [T][heads][d] (fp32, bf16 or fp16; views of any strides with unit stride along d) quantised into the slots
    [T] (int64; slot s is place s % page of page s / page) of a cache.  Slots outside the cache are not written; the
    others must differ from each other."""
    dt, T, heads, d, kt, kh = _head_rows(K, "K")
    vdt, vT, vheads, vd, vt, vh = _head_rows(V, "V")
    if (vdt, vT, vheads, vd) != (dt, T, heads, d):
        raise ValueError("K and V must agree in shape and dtype")
    pages, cheads, page = _cache(codes, scales, d)
    if cheads != heads:
        raise ValueError(f"the cache has {cheads} heads, K and V {heads}")
    _ints(slots, "slots", torch.int64, T)
    _one_device(codes, scales=scales, K=K, V=V, slots=slots)
    status = _lib.load().qamw_mxfp4_cache_write(K.data_ptr(), V.data_ptr(), dt, T, heads, d, kt, kh, vt, vh, slots.data_ptr(),
                                                codes.data_ptr(), scales.data_ptr(), pages, page, _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_cache_write", status)


def qamw_mxfp4_cache_read(codes: torch.Tensor, scales: torch.Tensor, slots: torch.Tensor, d: int, out_dtype=torch.float32,
                          K: Optional[torch.Tensor] = None, V: Optional[torch.Tensor] = None, stream=None):
    """(K, V) [T][heads][d]: the values in the slots [T] (int64) of a cache, in out_dtype (fp32, bf16 or fp16) or into given
    tensors of one dtype; 0 for a slot outside the cache."""
    pages, heads, page = _cache(codes, scales, d)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a GPU tensor [T]")
    T = slots.shape[0]
    _ints(slots, "slots", torch.int64, T)
    if K is not None or V is not None:
        out_dtype = (V if K is None else K).dtype
    if K is None:
        K = _empty_heads(T, heads, d, out_dtype, codes.device, stream)
    if V is None:
        V = _empty_heads(T, heads, d, out_dtype, codes.device, stream)
    dt, kT, kheads, kd, kt, kh = _head_rows(K, "K")
    vdt, vT, vheads, vd, vt, vh = _head_rows(V, "V")
    if (kT, kheads, kd) != (T, heads, d) or (vdt, vT, vheads, vd) != (dt, T, heads, d):
        raise ValueError("K and V must be [T][heads][d] of one dtype")
    _one_device(codes, scales=scales, K=K, V=V, slots=slots)
    status = _lib.load().qamw_mxfp4_cache_read(codes.data_ptr(), scales.data_ptr(), pages, page, heads, d, slots.data_ptr(), T,
                                               K.data_ptr(), V.data_ptr(), dt, kt, kh, vt, vh, _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_cache_read", status)
    return K, V


def qamw_mxfp4_cache_attention(Q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, table: torch.Tensor,
                               lengths: torch.Tensor, starts: Optional[torch.Tensor] = None, max_queries: Optional[int] = None,
                               scale: Optional[float] = None, causal: bool = True, window: int = 0, out_dtype=None,
                               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None):
    """(out, lse): attention of the queries Q [T][q_heads][d] over the cached tokens of their sequences.

    table [sequences][columns] int32 names the pages of each sequence, lengths [sequences] int32 its cached tokens, those
    of the queries among them.  Without starts every sequence has one query; with starts [sequences + 1] int32 sequence b
    has the queries starts[b] to starts[b + 1] - 1, its latest tokens.  max_queries: as many as any sequence has, which
    sizes the launch; of a sequence with more the first max_queries are computed.  T if not given: all of them in any
    case, in a launch and a workspace larger by the number of sequences.  causal: a query sees no token
    after its own; window > 0: only the latest `window` tokens up to its own.  scale: 1 / sqrt(d) if not given.
    out [T][q_heads][d] of out_dtype (that of Q if not given), lse [T][q_heads] fp32: 0 and -inf for a row that no token
    is left to; rows of queries that belong to no sequence stay as they were (in tensors made here: unset)."""
    qdt, T, q_heads, d, qt, qh = _head_rows(Q, "Q")
    pages, heads, page = _cache(codes, scales, d)
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be a GPU tensor [sequences][columns] with unit column stride")
    sequences, cols = table.shape
    pitch = table.stride(0) if sequences > 1 else cols
    if not table.is_cuda or table.dtype is not torch.int32:
        raise ValueError("table must be an int32 GPU tensor")
    _ints(lengths, "lengths", torch.int32, sequences)
    if starts is not None:
        _ints(starts, "starts", torch.int32, sequences + 1)
    if max_queries is None:
        max_queries = 1 if starts is None else max(T, 1)
    if out is None:
        out = _empty_heads(T, q_heads, d, Q.dtype if out_dtype is None else out_dtype, Q.device, stream)
    odt, oT, oheads, od, ot, oh = _head_rows(out, "out")
    if (oT, oheads, od) != (T, q_heads, d) or (out_dtype or out.dtype) != out.dtype:
        raise ValueError("out must be [T][q_heads][d] of out_dtype")
    if lse is None:
        lse = _empty((T, q_heads), torch.float32, Q.device, stream)
    elif lse.dtype is not torch.float32 or lse.shape != (T, q_heads) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [T][q_heads]")
    lib = _lib.load()
    if workspace is None:
        need = lib.qamw_mxfp4_cache_attention_workspace_bytes(T, sequences, max_queries, heads, q_heads, d, cols * page, qdt, odt)
        workspace = _workspace(need, Q.device, stream) if need else None
    else:
        _dev(workspace, "workspace")
    _one_device(Q, codes=codes, scales=scales, table=table, lengths=lengths, starts=starts, out=out, lse=lse, workspace=workspace)
    status = lib.qamw_mxfp4_cache_attention(
        Q.data_ptr(), qdt, T, q_heads, d, qt, qh, None if starts is None else starts.data_ptr(), sequences, max_queries,
        codes.data_ptr(), scales.data_ptr(), pages, page, heads, table.data_ptr(), cols, pitch, lengths.data_ptr(),
        d ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(), odt, ot, oh, lse.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes, _raw_stream(stream))
    if status:
        _lib.check("qamw_mxfp4_cache_attention", status)
    return out, lse
