"""Gradients of the norms for rows of more than 8192 values, over several rows
of every unit of the column sums, against oracle/norms.py (fp64).

Tolerances are those of the norms' other gradients.  mean(c v) is formed here
from three sums, of f dr, f g and f r (f = gate w_post y): each is off by (H +
4) 2^-24 of its terms' magnitudes, which together are those of c v, so that
(2 H + 16) 2^-24 of their mean holds as it does for the sum of c v itself.
"""

import ctypes

import numpy as np
import pytest

from oracle import norms

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}
U = 2.0 ** -24
TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)]
IDS = ["f16", "f16-f32", "bf16", "bf16-f32", "f32"]


def _np(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def _grad_tol(q, d_r, d_n, alpha, eps, post):
    T, H = d_n.shape
    one = np.ones((1, H))
    w_pre, w_post, gate = (q.get(k, one) for k in ("w_pre", "w_post", "gate"))
    a = 1 / norms.rms(q["r"], eps)
    b = 1 / norms.rms(q["y"], eps) if post else np.ones((T, 1))
    g, u, v = np.abs(d_n * w_pre), np.abs(q["r"] * a), np.abs(q["y"]) * b
    mag = np.abs(d_r) + a * (g + u * np.mean(g * u, axis=1, keepdims=True))
    e_dr = (2 * H + 16) * U * mag
    cols = lambda mags, errs: errs.sum(0) + T * U * mags.sum(0)
    c, e_c = mag * np.abs(gate * w_post), e_dr * np.abs(gate * w_post)
    m = np.mean(c * v, axis=1, keepdims=True)
    tol = {"d_residual": abs(alpha) * (e_dr + 2 * U * mag),
           "d_w_pre": cols(np.abs(d_n) * u, (H / 2 + 8) * U * np.abs(d_n) * u),
           "d_w_post": cols(mag * np.abs(gate) * v, (e_dr + (H / 2 + 8) * U * mag) * np.abs(gate) * v)}
    if post:
        em = np.mean(e_c * v, axis=1, keepdims=True) + (2 * H + 16) * U * m
        tol["d_y"] = b * (e_c + v * em + (H + 16) * U * (c + v * m))
    else:
        tol["d_y"] = e_c + 4 * U * c
    d, e = mag * v * np.abs(w_post), (e_dr + (H / 2 + 8) * U * mag) * v * np.abs(w_post)
    tol["d_gate"] = e if "gate" in q and q["gate"].ndim == 2 else cols(d, e)
    return tol


def _case(T, H, dtype, res_dtype, gate, post, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda dt, *s: torch.randn(s, generator=g, device="cuda").to(dt)
    v = dict(r=rand(res_dtype, T, H), y=rand(dtype, T, H), w_pre=rand(dtype, H))
    if post:
        v["w_post"] = rand(dtype, H)
    if gate != "none":
        v["gate"] = rand(dtype, *((H,) if gate == "vector" else (T, H)))
    return v, rand(res_dtype, T, H), rand(dtype, T, H)


def _check(got, v, d_r, d_n, alpha, post, what):
    q = {k: _np(t) for k, t in v.items()}
    ref = norms.block_norm_grad(q["r"], q["y"], _np(d_r), _np(d_n), q["w_pre"], q.get("w_post"), q.get("gate"), alpha, 1e-6, post)
    tol = _grad_tol(q, _np(d_r), _np(d_n), alpha, 1e-6, post)
    for k in got:
        out = _np(got[k])
        assert out.shape == ref[k].shape
        t = tol[k] * (1 + 2.0 ** -8) + np.abs(ref[k]) * (torch.finfo(got[k].dtype).eps / 2) * (1 + 2.0 ** -6) + TINY[got[k].dtype]
        bad = ~(np.abs(out - ref[k]) <= t)
        assert not bad.any(), (what, k, int(bad.sum()), float(np.nanmax(np.abs(out - ref[k]) / t)))


# runs of rows of one and of several; widths that end inside a workgroup's columns
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H,gate,post", [(1, 8193, "vector", True), (500, 8200, "token", True), (260, 12288, "vector", True),
                                           (300, 16384, "vector", True), (200, 16387, "none", True), (150, 20001, "token", False),
                                           (140, 32768, "vector", True), (2, 32767, "vector", False)])
def test_wide_gradients(T, H, gate, post, types):
    from bit_quantized_moe_token_amd import moeq
    v, d_r, d_n = _case(T, H, *types, gate, post, T + H)
    got = moeq.block_norm_grad(v["r"], d_n, v["y"], d_res=d_r, w_pre=v["w_pre"], w_post=v.get("w_post"), gate=v.get("gate"),
                               alpha=0.75, post_norm=post)
    assert set(got) == {"d_residual", "d_y", "d_w_pre"} | ({"d_w_post"} if post else set()) | ({"d_gate"} if gate != "none" else set())
    _check(got, v, d_r, d_n, 0.75, post, (T, H))
    again = moeq.block_norm_grad(v["r"], d_n, v["y"], d_res=d_r, w_pre=v["w_pre"], w_post=v.get("w_post"), gate=v.get("gate"),
                                 alpha=0.75, post_norm=post)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_wide_without_column_sums(types):
    """No weight's gradient wanted and a gate per token: no workspace."""
    from bit_quantized_moe_token_amd import _lib, moeq
    T, H = 9, 10001
    v, d_r, d_n = _case(T, H, *types, "token", True, 3)
    out = dict(d_residual=torch.empty_like(v["r"]), d_y=torch.empty_like(v["y"]), d_gate=torch.empty_like(v["y"]))
    p = lambda t: t.data_ptr()
    d = _lib.Norm(T, H, moeq._DTYPE[types[0]], moeq._DTYPE[types[1]], p(v["w_pre"]), p(v["w_post"]), p(v["gate"]), 1, 1, 0.75, 1e-6)
    st = _lib.lib().moeq_block_norm_grad(ctypes.byref(d), p(v["r"]), p(v["y"]), p(d_r), p(d_n), p(out["d_residual"]), p(out["d_y"]),
                                         None, None, p(out["d_gate"]), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    _check(out, v, d_r, d_n, 0.75, True, (T, H))


def test_wide_without_a_block():
    from bit_quantized_moe_token_amd import moeq
    g = torch.Generator(device="cuda").manual_seed(4)
    T, H = 270, 9000
    r, d_n, w = (torch.randn(s, generator=g, device="cuda").to(BF16) for s in ((T, H), (T, H), (H,)))
    got = moeq.block_norm_grad(r, d_n, w_pre=w)
    ref = norms.block_norm_grad(_np(r), None, np.zeros((T, H)), _np(d_n), _np(w), None, None, 1.0, 1e-6, True)
    a = 1 / norms.rms(_np(r), 1e-6)
    g_, u = np.abs(_np(d_n) * _np(w)), np.abs(_np(r) * a)
    mag = a * (g_ + u * np.mean(g_ * u, axis=1, keepdims=True))
    tol = {"d_residual": (2 * H + 16) * U * mag, "d_w_pre": ((H / 2 + 8 + T) * U * np.abs(_np(d_n)) * u).sum(0)}
    assert set(got) == set(ref)
    for k in ref:
        t = tol[k] * (1 + 2.0 ** -8) + np.abs(ref[k]) * (torch.finfo(got[k].dtype).eps / 2) * (1 + 2.0 ** -6) + TINY[got[k].dtype]
        assert (np.abs(_np(got[k]) - ref[k]) <= t).all(), k


def test_wide_gradients_captured_and_on_another_stream():
    """A captured pass, replayed with eager work between the replays, and a
    pass on another stream give the eager bits."""
    from bit_quantized_moe_token_amd import moeq
    v, d_r, d_n = _case(90, 9000, BF16, F32, "vector", True, 8)
    v["r"][3] *= 1e25                      # (a row whose sums are formed twice)

    def step():
        g = moeq.block_norm_grad(v["r"], d_n, v["y"], d_res=d_r, w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"], alpha=0.5)
        return [g[k] for k in sorted(g)]

    eager = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        assert all(torch.equal(a, b) for a, b in zip(step(), eager))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))
