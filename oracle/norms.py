"""Plain fp64 forms of the norms around a block and of their gradients
(numpy)."""

import numpy as np


def rms(v, eps):
    return np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def block_norm(res, y, w_pre, w_post, gate, alpha, eps, post_norm, rounded=lambda r: r):
    """(r', n); `rounded` gives r' as it is stored."""
    if y is None:
        r = res
    else:
        p = y / rms(y, eps) * (1.0 if w_post is None else w_post) if post_norm else y
        r = alpha * res + (1.0 if gate is None else gate) * p
    s = rounded(r)
    return r, s / rms(s, eps) * (1.0 if w_pre is None else w_pre)


def _through(grad, v, eps):
    """Gradient in v of v / rms(v), for the gradient `grad` of its result."""
    s = rms(v, eps)
    return grad / s - v * np.mean(grad * v, axis=1, keepdims=True) / s ** 3


def block_norm_grad(r, y, d_r, d_n, w_pre, w_post, gate, alpha, eps, post_norm):
    """Gradients of block_norm's inputs as a dict (r = its r')."""
    one = np.ones((1, r.shape[1]))
    wp, g = one if w_post is None else w_post, one if gate is None else gate
    out = {}
    dr = d_r + _through(d_n * (one if w_pre is None else w_pre), r, eps)
    if w_pre is not None:
        out["d_w_pre"] = (d_n * r / rms(r, eps)).sum(0)
    if y is None:
        out["d_residual"] = dr
        return out
    out["d_residual"] = alpha * dr
    unit = y / rms(y, eps) if post_norm else y
    out["d_y"] = _through(dr * g * wp, y, eps) if post_norm else dr * g
    if w_post is not None:
        out["d_w_post"] = (dr * g * unit).sum(0)
    if gate is not None:
        d = dr * unit * wp
        out["d_gate"] = d if gate.ndim == 2 else d.sum(0)
    return out
