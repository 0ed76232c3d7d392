"""Rows of routed tokens: the order by expert, the rows copied into it and combined again, with gradients.

Test infrastructure only (see ``oracle/__init__.py``). Pair p = t * top_k + j; ids outside 0 .. E - 1 have no expert.
Everything in FP64, pair by pair.
"""

import numpy as np


def sort(topk_ids, num_experts):
    """(row_of_pair int32 [T, top_k], pair_of_row int32 [P], offsets int32 [E + 1])."""
    ids = np.asarray(topk_ids)
    flat = ids.reshape(-1)
    row = np.full(flat.size, -1, dtype=np.int32)
    pair = np.full(flat.size, -1, dtype=np.int32)
    offsets = np.zeros(num_experts + 1, dtype=np.int32)
    r = 0
    for e in range(num_experts):
        offsets[e] = r
        for p in np.flatnonzero(flat == e):
            row[p] = r
            pair[r] = p
            r += 1
    offsets[num_experts] = r
    return row.reshape(ids.shape), pair, offsets


def permute(X, row_of_pair, Xs):
    """Xs with its named rows replaced."""
    Xs = np.array(Xs)
    for (t, _), r in np.ndenumerate(row_of_pair):
        if 0 <= r < Xs.shape[0]:
            Xs[r] = X[t]
    return Xs


def combine(Ys, row_of_pair, weights=None):
    T, top_k = row_of_pair.shape
    out = np.zeros((T, Ys.shape[1]))
    for (t, j), r in np.ndenumerate(row_of_pair):
        if 0 <= r < Ys.shape[0]:
            out[t] += (1.0 if weights is None else float(weights[t, j])) * Ys[r]
    return out


def combine_grad(dout, Ys, row_of_pair, weights, dYs):
    """(dYs with its named rows replaced, dweights)."""
    dYs = np.array(dYs, dtype=np.float64)
    dw = np.zeros(row_of_pair.shape)
    for (t, j), r in np.ndenumerate(row_of_pair):
        if 0 <= r < Ys.shape[0]:
            dYs[r] = float(weights[t, j]) * dout[t]
            dw[t, j] = np.dot(dout[t], Ys[r])
    return dYs, dw
