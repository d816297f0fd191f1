"""The 8-bit checkpoint format from its definition, in 64 bits (numpy)."""
from __future__ import annotations

import numpy as np


def pack(X):
    """(Q, S) of a float64 matrix: blocks of 32 along a row, S = 127 + floor(log2(max)),
    Q = x * 64 / 2^(S - 127) to nearest even, held in [-127, 127]; NaN blocks S = 255."""
    M, K = X.shape
    blocks = (K + 31) // 32
    Q, S = np.zeros((M, K), np.int8), np.zeros((M, blocks), np.uint8)
    for b in range(blocks):
        x = X[:, 32 * b:32 * b + 32]
        a = np.abs(x).max(1)
        ok = np.isfinite(a)
        e = np.frexp(np.where(ok, a, 0.0))[1] - 1
        s = np.where(a > 0, np.clip(e + 127, 0, 254), 0)
        q = np.rint(np.ldexp(np.where(ok[:, None], x, 0.0), (133 - s)[:, None]))
        Q[:, 32 * b:32 * b + 32] = np.clip(q, -127, 127).astype(np.int8)
        S[:, b] = np.where(ok, s, 255)
    return Q, S


def values(Q, S):
    """What (Q, S) stand for, in float64."""
    K = Q.shape[1]
    unit = np.where(S == 255, np.nan, np.ldexp(1.0, S.astype(np.int64) - 133))
    return Q.astype(np.float64) * np.repeat(unit, 32, axis=1)[:, :K]
