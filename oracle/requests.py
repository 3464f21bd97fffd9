"""Plain fp64 form of the low-rank adapters of many requests beside a shared
projection (numpy)."""

import numpy as np


def adapters(x, a, b, ids, y, scale=None, ranks=None):
    """(out [T, N], bound of what an error of one of z's relative size makes of
    it, magnitudes of its terms): y[r] + scale_i B_i (A_i x[r])."""
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    out = np.array(y, dtype=np.float64)
    worst, mag = np.zeros(out.shape), np.zeros(out.shape)
    n, R = a.shape[:2]
    for r, i in enumerate(ids):
        if not 0 <= i < n:
            continue
        rank = R if ranks is None else min(max(int(ranks[i]), 0), R)
        s = 1.0 if scale is None else float(scale[i])
        z = a[i, :rank] @ x[r]
        size = np.abs(a[i, :rank]) @ np.abs(x[r])
        out[r] += s * (b[i, :, :rank] @ z)
        worst[r] = abs(s) * np.abs(b[i, :, :rank]).sum(1) * (np.abs(z).max() if rank else 0.0)
        mag[r] = abs(s) * (np.abs(b[i, :, :rank]) @ size)
    return out, worst, mag


def adapters_of_many_rows(x, a, b, ids, y, scale=None, ranks=None):
    """adapters, one adapter after the other with all its rows."""
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    out = np.array(y, dtype=np.float64)
    worst, mag = np.zeros(out.shape), np.zeros(out.shape)
    n, R = a.shape[:2]
    for i in range(n):
        rows = np.flatnonzero(np.asarray(ids) == i)
        rank = R if ranks is None else min(max(int(ranks[i]), 0), R)
        s = 1.0 if scale is None else float(scale[i])
        A, B = a[i, :rank], b[i, :, :rank]
        z = x[rows] @ A.T
        out[rows] += s * (z @ B.T)
        worst[rows] = abs(s) * np.abs(B).sum(1) * np.abs(z).max(1, initial=0.0)[:, None]
        mag[rows] = abs(s) * (np.abs(x[rows]) @ np.abs(A).T @ np.abs(B).T)
    return out, worst, mag
