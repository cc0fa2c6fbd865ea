"""Vocabulary cross entropy and its gradient in plain NumPy (64 bits), from
the definition; shares no code with the kernels."""
from __future__ import annotations

import numpy as np


def counted(targets, V: int):
    targets = np.asarray(targets)
    return (targets >= 0) & (targets < V)


def forward(H, W, targets):
    """(loss [T], lse [T])."""
    H, W, targets = np.asarray(H, np.float64), np.asarray(W, np.float64), np.asarray(targets)
    T, V = H.shape[0], W.shape[0]
    z = H @ W.T
    m = z.max(axis=1) if T else np.zeros(0)
    lse = m + np.log(np.exp(z - m[:, None]).sum(axis=1))
    loss = np.zeros(T)
    for t in np.nonzero(counted(targets, V))[0]:
        loss[t] = lse[t] - z[t, targets[t]]
    return loss, lse


def logit_grad(H, W, targets, dloss):
    """G [T][V] = dloss_t (softmax - onehot); zero rows for tokens that are not counted."""
    H, W, targets = np.asarray(H, np.float64), np.asarray(W, np.float64), np.asarray(targets)
    T, V = H.shape[0], W.shape[0]
    G = np.zeros((T, V))
    for t in np.nonzero(counted(targets, V))[0]:
        z = W @ H[t]
        p = np.exp(z - z.max())
        p /= p.sum()
        p[targets[t]] -= 1.0
        G[t] = np.float64(dloss[t]) * p
    return G


def backward(H, W, targets, dloss):
    """(dH [T][d], dW [V][d]); the hidden state of a token that is not counted is not read."""
    H, W = np.asarray(H, np.float64), np.asarray(W, np.float64)
    G = logit_grad(H, W, targets, dloss)
    return G @ W, G.T @ np.where(counted(targets, W.shape[0])[:, None], H, 0.0)
