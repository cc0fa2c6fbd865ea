"""The attention cache in microscaled 4-bit floating point, in plain NumPy
(64 bits): layout, write, read and attention, token by token.

Written from the definitions; shares no code with the kernels."""
from __future__ import annotations

import numpy as np

from . import mxfp4 as M


def scale_bytes(d: int) -> int:
    nb = M.blocks(d)
    return next(n for n in (2, 4, 8) if n >= nb)


def new(pages: int, heads: int, page: int, d: int):
    return (np.zeros((2, pages, heads, page, M.row_bytes(d)), dtype=np.uint8),
            np.zeros((2, pages, heads, page, scale_bytes(d)), dtype=np.uint8))


def write(codes, scales, K, V, slots) -> None:
    """K and V [T][heads][d] into the slots, in place; slots outside the cache are passed over."""
    _, pages, heads, page, _ = codes.shape
    d, nb = K.shape[2], M.blocks(K.shape[2])
    for kv, x in enumerate((K, V)):
        c, s = M.quantize(np.asarray(x, dtype=np.float64).reshape(-1, d))
        c, s = c.reshape(-1, heads, c.shape[1]), s.reshape(-1, heads, s.shape[1])
        for t, slot in enumerate(slots):
            if 0 <= slot < pages * page:
                codes[kv, slot // page, :, slot % page] = c[t]
                scales[kv, slot // page, :, slot % page] = 0
                scales[kv, slot // page, :, slot % page, :nb] = s[t][:, :nb]


def _values(codes, scales, d):
    nb = M.blocks(d)
    flat = np.zeros((scales.size // scales.shape[-1], M.scale_bytes(d)), dtype=np.uint8)
    flat[:, :nb] = scales.reshape(-1, scales.shape[-1])[:, :nb]
    return M.dequantize(codes.reshape(-1, codes.shape[-1]), flat, d).reshape(*codes.shape[:-1], d)


def read(codes, scales, slots, d: int):
    """(K, V) [T][heads][d], 0 for slots outside the cache."""
    _, pages, heads, page, _ = codes.shape
    out = np.zeros((2, len(slots), heads, d))
    for t, slot in enumerate(slots):
        if 0 <= slot < pages * page:
            out[:, t] = _values(codes[:, slot // page, :, slot % page], scales[:, slot // page, :, slot % page], d)
    return out[0], out[1]


def attention(Q, codes, scales, table, lengths, starts, scale, causal=True, window=0):
    """(out, lse, weighted, plain) [T][q_heads]...: weighted is sum_t p_t |v_t| and plain sum_t |v_t|, the scales of
    the errors of out.  Rows of no sequence are NaN in all of them."""
    Q = np.asarray(Q, dtype=np.float64)
    T, q_heads, d = Q.shape
    _, pages, heads, page, _ = codes.shape
    group = q_heads // heads
    out, lse = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    weighted, plain = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan)
    for b, length in enumerate(lengths):
        n = int(starts[b + 1]) - int(starts[b])
        if n <= 0:
            continue
        length = max(0, min(int(length), table.shape[1] * page))
        pg = np.array([table[b, t // page] for t in range(length)], dtype=np.int64)
        held = (pg >= 0) & (pg < pages)
        at = np.where(held, pg, 0)
        off = np.arange(length) % page
        for h in range(heads):
            k = _values(codes[0, at, h, off], scales[0, at, h, off], d) if length else np.zeros((0, d))
            v = _values(codes[1, at, h, off], scales[1, at, h, off], d) if length else np.zeros((0, d))
            for i in range(n):
                place = length - n + i
                t = np.arange(length)
                sees = held.copy()
                if causal:
                    sees &= t <= place
                if window:
                    sees &= t > place - window
                row = starts[b] + i
                for j in range(h * group, (h + 1) * group):
                    if not sees.any():
                        out[row, j], lse[row, j], weighted[row, j], plain[row, j] = 0.0, -np.inf, 0.0, 0.0
                        continue
                    z = k[sees] @ Q[row, j] * scale
                    m = z.max()
                    p = np.exp(z - m)
                    lse[row, j] = m + np.log(p.sum())
                    p = p / p.sum()
                    # NaN times a weight, even one that has gone to 0, is NaN
                    out[row, j] = p @ v[sees]
                    weighted[row, j], plain[row, j] = p @ np.abs(v[sees]), np.abs(v[sees]).sum(axis=0)
    return out, lse, weighted, plain
