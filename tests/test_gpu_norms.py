"""Norms around a block and their gradients against oracle/norms.py (fp64).

Tolerances, per element, u = 2^-24 (half a step of fp32).  A sum of H fp32
terms in any order is off by at most H u of the sum of magnitudes; for sums
of squares that is H u relative, and half of it after the square root.  Each
value then takes a handful of roundings: forward 4 products and one sum for
r' (of the magnitudes alpha |res| and |gate p|), 3 for n; the result is
rounded once more to its type (half a step and half the smallest subnormal).
n is that of the r' that was stored, so the oracle norms the GPU's own r'.
Gradients: the same counted on magnitudes, see `_grad_tol`.
"""

import numpy as np
import pytest

from oracle import norms

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}
U = 2.0 ** -24


def _np(t):
    return None if t is None else t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def _round(ref, dtype):
    return np.abs(ref) * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def _close(got, ref, tol, what):
    got = _np(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the tolerance")


TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)]
IDS = ["f16", "f16-f32", "bf16", "bf16-f32", "f32"]
# one value, odd widths, every width class of the kernels and its borders
SIZES = [(1, 1), (5, 7), (3, 64), (9, 511), (4, 520), (2, 1024), (3, 1025), (17, 2048), (2, 2051), (3, 4096), (2, 4099),
         (2, 8192), (3, 8200), (1, 16384), (2, 16387), (1, 32768), (700, 130), (1100, 1032)]


def _inputs(T, H, dtype, res_dtype, gate, block, post, seed):
    rng = np.random.default_rng(seed)
    m = lambda dt, *s: torch.from_numpy(rng.standard_normal(s)).to(dt).cuda()
    v = dict(res=m(res_dtype, T, H), y=None, w_pre=m(dtype, H), w_post=None, gate=None)
    if block:
        v["y"] = m(dtype, T, H)
        if T > 2:
            v["y"][1] = 0                      # a block that gives nothing for a token
            v["res"][2] *= 2.0 ** -10
        if post:
            v["w_post"] = m(dtype, H)
        if gate != "none":
            v["gate"] = m(dtype, *((H,) if gate == "vector" else (T, H)))
    return v


def _forward(v, alpha, eps, post):
    from bit_quantized_moe_token_amd import moeq
    return moeq.block_norm(v["res"], v["y"], w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"], alpha=alpha, eps=eps,
                           post_norm=post)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_block_norm(i, types):
    T, H = SIZES[i]
    dtype, res_dtype = types
    block, post, gate = i % 5 != 4, i % 3 != 2, ("vector", "token", "none")[i % 3 if i < 12 else (i + 1) % 3]
    alpha, eps = (1.0, 0.75, -0.5)[i % 3], 1e-6
    v = _inputs(T, H, dtype, res_dtype, gate, block, post, i)
    r, n = _forward(v, alpha, eps, post)
    assert r.dtype == res_dtype and n.dtype == dtype
    q = {k: _np(a) for k, a in v.items()}
    ref, _ = norms.block_norm(q["res"], q["y"], q["w_pre"], q["w_post"], q["gate"], alpha, eps, post)
    if block:
        branch = ref - alpha * q["res"]
        tol = (H / 2 + 8) * U * np.abs(branch) + 2 * U * np.abs(alpha * q["res"]) + U * np.abs(ref)
        _close(r, ref, tol * (1 + 2.0 ** -10) + _round(ref, res_dtype) * (1 + 2.0 ** -7), f"r' {T}x{H}")
    else:
        assert r is v["res"]
    s = _np(r)
    ref_n = s / norms.rms(s, eps) * q["w_pre"]
    _close(n, ref_n, ((H / 2 + 8) * U * np.abs(ref_n)) * (1 + 2.0 ** -10) + _round(ref_n, dtype) * (1 + 2.0 ** -7), f"n {T}x{H}")


def _grad_tol(q, r, d_r, d_n, alpha, eps, post, H, T):
    """Bounds on the fp32 error of every gradient before its last rounding.
    dr = d_r + a (g - u mean(g u)): a carries (H/2 + 4) u, the mean (H + 4) u
    of mean |g u|, the rest 6 roundings, all of the terms' magnitudes."""
    one = np.ones((1, H))
    w_pre, w_post, gate = (one if q[k] is None else q[k] for k in ("w_pre", "w_post", "gate"))
    a = 1 / norms.rms(r, eps)
    g, u = np.abs(d_n * w_pre), np.abs(r * a)
    mag = np.abs(d_r) + a * (g + u * np.mean(g * u, axis=1, keepdims=True))
    e_dr = (2 * H + 16) * U * mag
    tol = {"d_residual": abs(alpha) * (e_dr + 2 * U * mag) if q["y"] is not None else e_dr}
    cols = lambda mags, errs: errs.sum(0) + T * U * mags.sum(0)
    tol["d_w_pre"] = cols(np.abs(d_n) * u, (H / 2 + 8) * U * np.abs(d_n) * u)
    if q["y"] is None:
        return tol
    b = 1 / norms.rms(q["y"], eps) if post else np.ones((len(r), 1))
    v = np.abs(q["y"]) * b
    c, e_c = mag * np.abs(gate * w_post), e_dr * np.abs(gate * w_post)
    if post:
        m = np.mean(c * v, axis=1, keepdims=True)
        em = np.mean(e_c * v, axis=1, keepdims=True) + (2 * H + 16) * U * m
        tol["d_y"] = b * (e_c + v * em + (H + 16) * U * (c + v * m))
    else:
        tol["d_y"] = e_c + 4 * U * c
    tol["d_w_post"] = cols(mag * np.abs(gate) * v, (e_dr + (H / 2 + 8) * U * mag) * np.abs(gate) * v)
    d, e = mag * v * np.abs(w_post), (e_dr + (H / 2 + 8) * U * mag) * v * np.abs(w_post)
    tol["d_gate"] = e if q["gate"] is not None and q["gate"].ndim == 2 else cols(d, e)
    return tol


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_block_norm_grad(i, types):
    from bit_quantized_moe_token_amd import moeq
    T, H = SIZES[i]
    dtype, res_dtype = types
    block, post, gate = i % 5 != 4, i % 3 != 2, ("vector", "token", "none")[i % 3 if i < 12 else (i + 1) % 3]
    alpha, eps = (1.0, 0.75, -0.5)[i % 3], 1e-6
    v = _inputs(T, H, dtype, res_dtype, gate, block, post, 50 + i)
    rng = np.random.default_rng(90 + i)
    d_r = torch.from_numpy(rng.standard_normal((T, H))).to(res_dtype).cuda() if i % 4 else None
    d_n = torch.from_numpy(rng.standard_normal((T, H))).to(dtype).cuda()
    got = moeq.block_norm_grad(v["res"], d_n, v["y"], d_res=d_r, w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"],
                               alpha=alpha, eps=eps, post_norm=post)
    q = {k: _np(a) for k, a in v.items()}
    dr = _np(d_r) if d_r is not None else np.zeros((T, H))
    ref = norms.block_norm_grad(q["res"], q["y"], dr, _np(d_n), q["w_pre"], q["w_post"], q["gate"], alpha, eps, post)
    tol = _grad_tol(q, q["res"], dr, _np(d_n), alpha, eps, post, H, T)
    assert set(got) == set(ref)
    for k in ref:
        _close(got[k], ref[k], tol[k] * (1 + 2.0 ** -8) + _round(np.abs(ref[k]), got[k].dtype) * (1 + 2.0 ** -6), f"{k} {T}x{H}")
    want = {"d_residual": res_dtype, "d_y": dtype, "d_w_pre": F32, "d_w_post": F32, "d_gate": dtype if gate == "token" else F32}
    assert all(got[k].dtype == want[k] for k in got)


def test_in_place_and_unaligned():
    """res_out = residual and n = y, and rows that start at odd elements."""
    from bit_quantized_moe_token_amd import moeq
    for T, H in ((3, 4096), (4, 77), (1, 20000)):
        v = _inputs(T, H, BF16, BF16, "vector", True, True, H)
        r, n = _forward(v, 0.75, 1e-6, True)
        odd = {}
        for k, t in v.items():
            buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            odd[k] = buf[1:].view(t.shape).copy_(t)
        r2, n2 = moeq.block_norm(odd["res"], odd["y"], w_pre=odd["w_pre"], w_post=odd["w_post"], gate=odd["gate"], alpha=0.75,
                                 eps=1e-6, res_out=odd["res"], n_out=odd["y"])
        assert r2 is odd["res"] and n2 is odd["y"]
        assert torch.equal(r, r2) and torch.equal(n, n2)


def test_bad_rows_stay_alone():
    v = _inputs(6, 300, F16, F32, "vector", True, True, 0)
    v["y"][3, 5] = float("nan")
    v["res"][4, 0] = float("inf")
    r, n = _forward(v, 1.0, 1e-6, True)
    ok = torch.isfinite(n).all(1).cpu().tolist()
    assert ok == [True, True, True, False, False, True]


def test_no_tokens():
    from bit_quantized_moe_token_amd import moeq
    e = torch.empty((0, 64), dtype=F16, device="cuda")
    w = torch.ones(64, dtype=F16, device="cuda")
    r, n = moeq.block_norm(e, e, w_pre=w, w_post=w, gate=w)
    assert r.shape == n.shape == (0, 64)
    g = moeq.block_norm_grad(e, e, e, w_pre=w, w_post=w, gate=w)
    assert all(float(g[k].abs().sum()) == 0 and g[k].shape == (64,) for k in ("d_w_pre", "d_w_post", "d_gate"))


def test_refusals():
    from bit_quantized_moe_token_amd import moeq
    v = _inputs(4, 64, F16, F32, "vector", True, True, 0)
    kw = dict(w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"])
    with pytest.raises(ValueError):
        moeq.block_norm(v["res"], v["y"][:3], **kw)
    with pytest.raises(TypeError):
        moeq.block_norm(v["res"], v["y"].float(), **kw)
    with pytest.raises(ValueError):
        moeq.block_norm(v["res"].T.contiguous().T, v["y"], **kw)
    with pytest.raises(ValueError):
        moeq.block_norm(v["res"], v["y"], w_pre=v["w_pre"][:63])
    with pytest.raises(TypeError):
        moeq.block_norm(v["res"].cpu(), v["y"], **kw)
    with pytest.raises(moeq.MoeqError):
        moeq.block_norm(v["res"], v["y"], eps=0.0, **kw)
    with pytest.raises(moeq.MoeqError):
        moeq.block_norm(v["res"], v["y"], post_norm=False, **kw)
    with pytest.raises(ValueError):
        moeq.block_norm(v["res"], w_pre=v["w_pre"], res_out=v["res"])


def test_graph_and_stream():
    from bit_quantized_moe_token_amd import moeq
    v = _inputs(333, 1536, BF16, F32, "vector", True, True, 1)
    d_n, d_r = torch.randn(333, 1536, device="cuda").to(BF16), torch.randn(333, 1536, device="cuda")
    kw = dict(w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"], alpha=0.5)

    def step():
        r, n = moeq.block_norm(v["res"], v["y"], **kw)
        g = moeq.block_norm_grad(r, d_n, v["y"], d_res=d_r, **kw)
        return [r, n] + [g[k] for k in sorted(g)]

    eager = [t.clone() for t in step()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        assert all(torch.equal(a, b) for a, b in zip(step(), eager))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_rows_beyond_32_bit_offsets():
    """Rows whose elements lie behind 2^31 come out as in a call of their own
    (of enough rows for the same variant of the kernel)."""
    from bit_quantized_moe_token_amd import moeq
    H, T = 8192, 2 ** 18 + 40
    gen = torch.Generator(device="cuda").manual_seed(9)
    few = lambda: torch.randn((64, H), generator=gen, device="cuda").to(BF16)
    many = lambda t: t.repeat(T // 64 + 1, 1)[:T].contiguous()
    res, y, gate, d_n = few(), few(), few(), few()
    w = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(BF16)
    last = [(T - 1 - i) % 64 for i in range(300)]
    r, n = moeq.block_norm(many(res), many(y), w_pre=w, w_post=w, gate=many(gate), alpha=0.5)
    r0, n0 = moeq.block_norm(res[last], y[last], w_pre=w, w_post=w, gate=gate[last], alpha=0.5)
    assert torch.equal(r[-300:].flip(0), r0) and torch.equal(n[-300:].flip(0), n0)
    del n
    g = moeq.block_norm_grad(r, many(d_n), many(y), w_pre=w, w_post=w, gate=many(gate), alpha=0.5)
    g0 = moeq.block_norm_grad(r0, d_n[last], y[last], w_pre=w, w_post=w, gate=gate[last], alpha=0.5)
    for name in ("d_residual", "d_y", "d_gate"):
        assert torch.equal(g[name][-300:].flip(0), g0[name]), name
    del g
    q, s = moeq.quantize_i8(r)
    q0, s0 = moeq.quantize_i8(r0)
    assert torch.equal(q[-300:].flip(0), q0) and torch.equal(s[-300:].flip(0), s0)
