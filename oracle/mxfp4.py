"""Microscaled 4-bit floating point in plain NumPy (64 bits): blocks of 32
with one power-of-two scale, elements of magnitude {0, .5, 1, 1.5, 2, 3, 4, 6}.

Written from the format's definition; shares no code with the kernels."""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(d: int) -> int:
    return -(-d // BLOCK)


def row_bytes(d: int) -> int:
    return 16 * blocks(d)


def scale_bytes(d: int) -> int:
    return -(-blocks(d) // 16) * 16


def element(a: float) -> int:
    """Index of the magnitude nearest to a >= 0; a tie goes to the even index; beyond 6 to 6."""
    dist = [abs(a - m) for m in MAGNITUDES]
    best = min(dist)
    near = [i for i, x in enumerate(dist) if x == best]
    return next((i for i in near if i % 2 == 0), near[0])


def quantize(W):
    """W [N][d] -> (codes [N][row_bytes], scales [N][scale_bytes]) uint8."""
    W = np.asarray(W, dtype=np.float64)
    N, d = W.shape
    nb = blocks(d)
    full = np.zeros((N, nb * BLOCK))
    full[:, :d] = W
    full = full.reshape(N, nb, BLOCK)
    scales = np.zeros((N, scale_bytes(d)), dtype=np.uint8)
    nib = np.zeros((N, nb, BLOCK), dtype=np.uint8)
    finite = np.isfinite(full).all(axis=2)
    m = np.abs(np.where(np.isfinite(full), full, 0.0)).max(axis=2)
    # frexp: m = f 2^x with f in [1/2, 1), so floor(log2 m) = x - 1
    e = np.where(m > 0, np.maximum(np.frexp(m)[1] - 1 - 2, -127), -127)
    scales[:, :nb] = np.where(finite, e + 127, 255)
    a = np.ldexp(np.abs(np.where(np.isfinite(full), full, 0.0)), -e[:, :, None])
    dist = np.abs(a[..., None] - MAGNITUDES)
    # even indices first: argmin keeps the first of equal distances
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    idx = order[np.argmin(dist[..., order], axis=-1)]
    nib[...] = idx | (np.signbit(full).astype(np.uint8) << 3)
    nib[~finite] = 0
    nib = nib.reshape(N, -1)
    return (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8), scales


def dequantize(codes, scales, d: int):
    """The [N][d] values, float64; NaN in blocks of scale 255."""
    codes = np.asarray(codes)
    nb = blocks(d)
    nib = np.stack([codes & 15, codes >> 4], axis=2).reshape(codes.shape[0], nb, BLOCK)
    mag = MAGNITUDES[nib & 7]
    code = np.asarray(scales)[:, :nb].astype(np.int64)[:, :, None]
    val = np.ldexp(np.where(nib >= 8, -mag, mag), code - 127)
    val = np.where(code == 255, np.nan, val)
    return val.reshape(codes.shape[0], -1)[:, :d]


def matmul(X, codes, scales):
    """(Y, sum of |products|): the quantised X times the decoded matrix, float64."""
    d = np.asarray(X).shape[1]
    Xq = dequantize(*quantize(X), d)
    W = dequantize(codes, scales, d)
    return Xq @ W.T, np.abs(Xq) @ np.abs(W).T


def adapter_matmul(X, codes, scales, A, B, index, factors):
    """(Y, sum of |products| of the first term, of the second, sum of |U| |B|): the product plus the adapters of the
    tokens' own, float64."""
    X = np.asarray(X, dtype=np.float64)
    Y, S = matmul(X, codes, scales)
    extra, inner = np.zeros_like(Y), np.zeros_like(Y)
    for t, i in enumerate(index):
        if 0 <= i < len(A):
            u = factors[i] * (A[i] @ X[t])
            Y[t] += B[i] @ u
            extra[t] = np.abs(B[i]) @ (abs(factors[i]) * (np.abs(A[i]) @ np.abs(X[t])))
            inner[t] = np.abs(B[i]) @ np.abs(u)
    return Y, S, extra, inner
