"""W8A8: INT8 weights with one scale per output channel, INT8 activations with one scale per row.

Test infrastructure only (see ``oracle/__init__.py``).

The scale and the codes are decided in IEEE FP32 (as in ``oracle.w4a8``, with the whole row as the block):
s = amax / 127, xq = clamp(rint(x / s), -127, 127); an all-zero row has s = 0 and xq = 0; a row with a NaN or an
infinity has that as s and xq = 0. The product is Y[m][n] = sx[m] sw[n] I[m][n] with the exact integer sum I.
"""

import numpy as np

F32 = np.float32


def quantize_rows(X):
    """X [M, K] (float32 values of the inputs) -> (xq int8 [M, K], s float32 [M])."""
    X = np.asarray(X)
    if X.dtype != np.float32:
        raise TypeError("X must be float32 (the exact values of the inputs)")
    amax = np.abs(X).max(axis=1)  # NaN if the row has one
    s = (amax / F32(127.0)).astype(np.float32)
    usable = np.isfinite(s) & (s > 0)
    safe = np.where(usable, s, F32(1.0)).astype(np.float32)
    finite = np.where(usable[:, None], X, F32(0.0))
    xq = np.clip(np.rint((finite / safe[:, None]).astype(np.float32)), -127, 127)
    return xq.astype(np.int8), s


def quantize_weight(W):
    """W float32 [K, N] -> (wq int8 [N, K], sw float32 [N])."""
    return quantize_rows(np.ascontiguousarray(np.asarray(W).T))


def integer_sums(xq, wq):
    """I[m][n] = sum_k xq[m][k] wq[n][k], exact. (FP64 products: every partial sum is below 2^53.)"""
    return np.asarray(xq).astype(np.float64) @ np.asarray(wq).astype(np.float64).T


def matmul(xq, sx, wq, sw):
    """Y in FP64."""
    return integer_sums(xq, wq) * np.asarray(sx, dtype=np.float64)[:, None] * np.asarray(sw, dtype=np.float64)[None, :]


def routed_matmul(xq, sx, offsets, wq, sw):
    """Y in FP64 for rows sorted by expert, NaN in rows of no expert's run."""
    Y = np.full((xq.shape[0], wq.shape[1]), np.nan)
    for e in range(wq.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            Y[a:b] = matmul(xq[a:b], sx[a:b], wq[e], sw[e])
    return Y
