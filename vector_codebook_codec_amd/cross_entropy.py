"""Vocabulary cross entropy and its gradient over torch device tensors
(include/qamw.h states the formulas); the T x V logits are never stored."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .codec import _WDT, _dev, _empty, _matrix, _raw_stream, _vec, _workspace

__all__ = [
    "qamw_cross_entropy",
    "qamw_cross_entropy_grad",
    "qamw_cross_entropy_grad_workspace_bytes",
    "qamw_cross_entropy_workspace_bytes",
]


def qamw_cross_entropy_workspace_bytes(T: int, V: int, d: int, dtype=torch.bfloat16) -> int:
    return int(_lib.load().qamw_cross_entropy_workspace_bytes(T, V, d, _WDT[dtype]))


def qamw_cross_entropy_grad_workspace_bytes(T: int, V: int, d: int, dtype=torch.bfloat16) -> int:
    return int(_lib.load().qamw_cross_entropy_grad_workspace_bytes(T, V, d, _WDT[dtype]))


def _head(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor):
    T, d, ldh = _matrix(H, "H")
    V, d2, ldw = _matrix(W, "W")
    if d2 != d:
        raise ValueError("H [T][d] and W [V][d] must agree")
    if H.dtype not in _WDT or W.dtype != H.dtype:
        raise ValueError("H and W must both be float32 or both bfloat16")
    _vec(targets, "targets", T, torch.int64)
    return T, V, d, ldh, ldw


def qamw_cross_entropy(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, loss: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """(loss [T], lse [T]) fp32: loss_t = lse_t - <H_t, W_targets[t]> with lse_t = log sum_v exp <H_t, W_v>; 0 for a
    token whose target is outside [0, V)."""
    T, V, d, ldh, ldw = _head(H, W, targets)
    if loss is None:
        loss = _empty(T, torch.float32, H.device, stream)
    if lse is None:
        lse = _empty(T, torch.float32, H.device, stream)
    _vec(loss, "loss", T)
    _vec(lse, "lse", T)
    lib = _lib.load()
    dt = _WDT[H.dtype]
    if workspace is None:
        workspace = _workspace(lib.qamw_cross_entropy_workspace_bytes(T, V, d, dt), H.device, stream)
    else:
        _dev(workspace, "workspace")
    _lib.check("qamw_cross_entropy", lib.qamw_cross_entropy(
        H.data_ptr(), dt, T, d, ldh, W.data_ptr(), V, ldw, targets.data_ptr(), loss.data_ptr(), lse.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _raw_stream(stream)))
    return loss, lse


def qamw_cross_entropy_grad(H: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                            dloss: torch.Tensor, dH: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                            need_dH: bool = True, need_dW: bool = True, workspace: Optional[torch.Tensor] = None,
                            stream=None):
    """(dH [T][d], dW [V][d]) in H's dtype from the loss's upstream gradient dloss [T] and qamw_cross_entropy's lse;
    None in the place of one that is not needed (a frozen head, say)."""
    T, V, d, ldh, ldw = _head(H, W, targets)
    _vec(lse, "lse", T)
    _vec(dloss, "dloss", T)
    if dH is None and need_dH:
        dH = _empty((T, d), H.dtype, H.device, stream)
    if dW is None and need_dW:
        dW = _empty((V, d), H.dtype, H.device, stream)
    lddh = lddw = d
    if dH is not None:
        n2, d2, lddh = _matrix(dH, "dH")
        if (n2, d2) != (T, d) or dH.dtype != H.dtype:
            raise ValueError("dH must be T x d of H's dtype")
    if dW is not None:
        n2, d2, lddw = _matrix(dW, "dW")
        if (n2, d2) != (V, d) or dW.dtype != H.dtype:
            raise ValueError("dW must be V x d of H's dtype")
    lib = _lib.load()
    dt = _WDT[H.dtype]
    if workspace is None:
        workspace = _workspace(lib.qamw_cross_entropy_grad_workspace_bytes(T, V, d, dt), H.device, stream)
    _dev(workspace, "workspace")
    _lib.check("qamw_cross_entropy_grad", lib.qamw_cross_entropy_grad(
        H.data_ptr(), dt, T, d, ldh, W.data_ptr(), V, ldw, targets.data_ptr(), lse.data_ptr(), dloss.data_ptr(),
        None if dH is None else dH.data_ptr(), lddh, None if dW is None else dW.data_ptr(), lddw,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(stream)))
    return dH, dW
