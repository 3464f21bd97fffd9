"""Plain fp64 forms of the products of expert-sorted rows with one matrix per
expert, of their gradients and of the 8-bit coding of rows (numpy)."""

import numpy as np


def source_rows(P, T, pairs=None, k=1):
    """Source row of every sorted row; -1 where it lies outside [0, T)."""
    src = np.arange(P) if pairs is None else np.where(np.asarray(pairs) >= 0, np.asarray(pairs) // k, -1)
    return np.where((src >= 0) & (src < T), src, -1)


def gather(x, src):
    """Rows x[src] in fp64, zeros for src = -1."""
    out = np.zeros((len(src), x.shape[1]))
    ok = src >= 0
    out[ok] = np.asarray(x, dtype=np.float64)[src[ok]]
    return out


def grouped(x, w, offsets, src, y0):
    """y0 (fp64 [P, N]) with the rows of every expert e replaced by
    x[src[r]] . w[e]^T; w [E, N, K]."""
    y = np.array(y0, dtype=np.float64)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            y[lo:hi] = gather(x, src[lo:hi]) @ np.asarray(w[e], dtype=np.float64).T
    return y


def wgrad(dy, x, offsets, src):
    """[E, N, K]: the sum over each expert's rows of dy[r] x[src[r]]^T."""
    E = len(offsets) - 1
    out = np.zeros((E, dy.shape[1], x.shape[1]))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        out[e] = np.asarray(dy[lo:hi], dtype=np.float64).T @ gather(x, src[lo:hi])
    return out


def code_i8(x):
    """(codes int8, scales fp32) of the rows of x (fp32 [rows, cols]): every
    quotient rounded to fp32."""
    x = np.asarray(x, dtype=np.float32)
    codes = np.zeros(x.shape, dtype=np.int8)
    scales = np.ones(x.shape[0], dtype=np.float32)
    for r in range(x.shape[0]):
        a = np.max(np.abs(x[r])) if x.shape[1] else np.float32(0)
        if not np.all(np.isfinite(x[r])):
            scales[r] = np.nan
        elif a >= np.float32(2.0 ** -118):
            scales[r] = a / np.float32(127)
            codes[r] = np.rint(x[r] / scales[r]).astype(np.int8)
    return codes, scales
