"""Norms of many rows against oracle/norms.py (fp64): the variants for more
than 256 tokens, and gradients where a unit of the column sums takes several
rows, of every width class.

Tolerances as in the norms' other tests.  Of the column sums they are bounds
on every order of summing T fp32 terms.
"""

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


def _close(got, ref, tol, what):
    got = _np(got)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)), np.argwhere(bad)[0])


def _rounding(ref, dtype):
    return np.abs(ref) * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def _case(T, H, dtype, res_dtype, gate, post, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda dt, *s: torch.randn(s, generator=g, device="cuda").to(dt)
    v = dict(r=rand(res_dtype, T, H), y=rand(dtype, T, H), w_pre=rand(dtype, H))
    if post:
        v["w_post"] = rand(dtype, H)
    if gate != "none":
        v["gate"] = rand(dtype, *((H,) if gate == "vector" else (T, H)))
    return v, rand


# each side of the switch at 256 tokens, widths that fill the threads and that do not
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H", [(256, 4096), (257, 4096), (257, 2049), (300, 2051), (259, 4095), (256, 4099), (257, 4099),
                                 (257, 8192), (300, 8191), (257, 6000), (1030, 512), (1030, 1000), (520, 2048), (300, 16384),
                                 (258, 20001)])
@pytest.mark.parametrize("gate", ["vector", "token"])
def test_block_norm_of_many_rows(T, H, gate, types):
    from bit_quantized_moe_token_amd import moeq
    dtype, res_dtype = types
    v, _ = _case(T, H, dtype, res_dtype, gate, True, T + H)
    r, n = moeq.block_norm(v["r"], v["y"], w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"], alpha=0.75)
    q = {k: _np(t) for k, t in v.items()}
    ref, _ = norms.block_norm(q["r"], q["y"], q["w_pre"], q["w_post"], q["gate"], 0.75, 1e-6, True)
    branch = ref - 0.75 * q["r"]
    tol = (H / 2 + 8) * U * np.abs(branch) + 2 * U * np.abs(0.75 * q["r"]) + U * np.abs(ref)
    _close(r, ref, tol * (1 + 2.0 ** -10) + _rounding(ref, res_dtype) * (1 + 2.0 ** -7), "r'")
    s = _np(r)
    ref = s / norms.rms(s, 1e-6) * q["w_pre"]
    _close(n, ref, (H / 2 + 8) * U * np.abs(ref) * (1 + 2.0 ** -10) + _rounding(ref, dtype) * (1 + 2.0 ** -7), "n")


def _grad_tol(q, d_r, d_n, alpha, eps):
    T, H = d_n.shape
    a, b = 1 / norms.rms(q["r"], eps), 1 / norms.rms(q["y"], eps)
    w_pre, w_post, gate = q["w_pre"], np.abs(q["w_post"]), np.abs(q["gate"])
    g, u, v = np.abs(d_n * w_pre), np.abs(q["r"] * a), np.abs(q["y"]) * b
    mag = np.abs(d_r) + a * (g + u * np.mean(g * u, axis=1, keepdims=True))
    e_dr = (2 * H + 16) * U * mag
    cols = lambda mags, errs: errs.sum(0) + T * U * mags.sum(0)
    c, e_c = mag * gate * w_post, e_dr * gate * w_post
    m = np.mean(c * v, axis=1, keepdims=True)
    em = np.mean(e_c * v, axis=1, keepdims=True) + (2 * H + 16) * U * m
    d, e = mag * v * w_post, (e_dr + (H / 2 + 8) * U * mag) * v * w_post
    return {"d_residual": abs(alpha) * (e_dr + 2 * U * mag),
            "d_w_pre": cols(np.abs(d_n) * u, (H / 2 + 8) * U * np.abs(d_n) * u),
            "d_w_post": cols(mag * gate * v, (e_dr + (H / 2 + 8) * U * mag) * gate * v),
            "d_y": b * (e_c + v * em + (H + 16) * U * (c + v * m)),
            "d_gate": e if gate.ndim == 2 else cols(d, e)}


# several rows of every unit: T above 4096 units of 64 threads, 2048, 1024, 512 and 256 of the next widths, 204 to 64 of the widest
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H", [(9000, 64), (9001, 401), (4500, 1000), (2100, 2048), (1100, 1032), (1700, 4096), (1100, 3001),
                                 (900, 8192), (600, 8191), (530, 8193), (400, 16384), (200, 32768)])
@pytest.mark.parametrize("gate", ["vector", "token"])
def test_gradients_of_many_rows(T, H, gate, types):
    from bit_quantized_moe_token_amd import moeq
    dtype, res_dtype = types
    v, rand = _case(T, H, dtype, res_dtype, gate, True, T + H)
    d_r, d_n = rand(res_dtype, T, H), rand(dtype, T, H)
    got = moeq.block_norm_grad(v["r"], d_n, v["y"], d_res=d_r, w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"], alpha=0.75)
    q = {k: _np(t) for k, t in v.items()}
    ref = norms.block_norm_grad(q["r"], q["y"], _np(d_r), _np(d_n), q["w_pre"], q["w_post"], q["gate"], 0.75, 1e-6, True)
    tol = _grad_tol(q, _np(d_r), _np(d_n), 0.75, 1e-6)
    assert set(got) == set(ref)
    for k in ref:
        _close(got[k], ref[k], tol[k] * (1 + 2.0 ** -8) + _rounding(ref[k], got[k].dtype) * (1 + 2.0 ** -6), k)


def test_column_sums_of_rows_beyond_32_bit_offsets():
    """d_w_pre and d_w_post of 64 rows repeated past 2^31 elements: as many
    times the sums over the 64 (in fp64)."""
    from bit_quantized_moe_token_amd import moeq
    H, reps = 8192, 4097
    T = 64 * reps
    g = torch.Generator(device="cuda").manual_seed(9)
    few = lambda: torch.randn((64, H), generator=g, device="cuda").to(BF16)
    r, y, gate, d_n = few(), few(), few(), few()
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    got = moeq.block_norm_grad(r.repeat(reps, 1), d_n.repeat(reps, 1), y.repeat(reps, 1), w_pre=w, w_post=w,
                               gate=gate.repeat(reps, 1), alpha=0.5)
    q = dict(r=_np(r), y=_np(y), gate=_np(gate), w_pre=_np(w), w_post=_np(w))
    zero = np.zeros((64, H))
    ref = norms.block_norm_grad(q["r"], q["y"], zero, _np(d_n), q["w_pre"], q["w_post"], q["gate"], 0.5, 1e-6, True)
    tol = _grad_tol(q, zero, _np(d_n), 0.5, 1e-6)
    # per repetition the 64 rows' own error; T 2^-24 of the magnitudes for the sum over all (64 2^-24 of it is in tol)
    for k in ("d_w_pre", "d_w_post"):
        _close(got[k], reps * ref[k], reps * reps * tol[k] * (1 + 2.0 ** -8) + _rounding(reps * ref[k], F32), k)
