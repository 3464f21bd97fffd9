"""Rows of very large and very small magnitudes against the fp64 forms.

A row's scale drops out of its norm, so what a sum of squares loses to the
range of fp32 is lost from the result: rows of bf16 and fp32 values from about
2^64 on, and rows whose squares vanish where eps is as small.  Tolerances are
those of the norms' own tests, with 2 roundings more for the scaled sum; a
result of fp32 arithmetic below 2^-126 is off by another 2^-150 for every
step (at most 16 here).
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
    assert got.shape == ref.shape and np.isfinite(ref).all(), what
    bad = ~(np.abs(got - ref) <= tol + 16 * 2.0 ** -150)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the tolerance, first at "
                           f"{np.argwhere(bad)[0]}")


# (magnitude of the block's rows, of the residual's, eps)
MAGNITUDES = [(1e20, 1.0, 1e-6), (1.0, 1e20, 1e-6), (1e20, 1e20, 1e-6), (1e-20, 1e-20, 1e-6), (1e-20, 1e-20, 1e-38),
              (1e-20, 1e-20, 1e-42), (1e36, 1e36, 1e-6), (1e18, 1e18, 1e-6), (1.0, 1e-20, 1e-30), (1e20, 1e20, 1e29)]
# every width class of the kernels
WIDTHS = [1, 7, 64, 520, 1030, 4096, 8192, 16384, 20000]


def _rows(rng, T, H, scale, dtype):
    """Normal values times `scale`; row 1 zeros but for one value, row 2 a
    mixture of scales, where there are such rows."""
    v = rng.standard_normal((T, H)) * scale
    if T > 2:
        v[1, : H - 1] = 0
        v[2] *= np.where(rng.random(H) < 0.5, 1.0, 1e-10)
    return torch.from_numpy(v).to(dtype).cuda()


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("m", range(len(MAGNITUDES)))
def test_block_norm_of_any_magnitude(m, types):
    from bit_quantized_moe_token_amd import moeq
    dtype, res_dtype = types
    my, mr, eps = MAGNITUDES[m]
    eps = float(np.float32(eps))
    for H in WIDTHS:
        rng = np.random.default_rng(1000 * m + H)
        T = 3 if H > 1 else 1
        y, res = _rows(rng, T, H, my, dtype), _rows(rng, T, H, mr, res_dtype)
        w, q = (torch.from_numpy(1 + 0.2 * rng.standard_normal(H)).to(dtype).cuda() for _ in range(2))
        r, n = moeq.block_norm(res, y, w_pre=w, w_post=q, alpha=0.75, eps=eps)
        ref, _ = norms.block_norm(_np(res), _np(y), _np(w), _np(q), None, 0.75, eps, True)
        branch = ref - 0.75 * _np(res)
        tol = (H / 2 + 10) * U * np.abs(branch) + 2 * U * np.abs(0.75 * _np(res)) + U * np.abs(ref)
        _close(r, ref, tol * (1 + 2.0 ** -10) + _round(ref, res_dtype) * (1 + 2.0 ** -7), f"r' {T}x{H}")
        s = _np(r)
        ref_n = s / norms.rms(s, eps) * _np(w)
        _close(n, ref_n, (H / 2 + 10) * U * np.abs(ref_n) * (1 + 2.0 ** -10) + _round(ref_n, dtype) * (1 + 2.0 ** -7), f"n {T}x{H}")
        # without a block, on the same residual
        _, n = moeq.block_norm(res, w_pre=w, eps=eps)
        s = _np(res)
        ref_n = s / norms.rms(s, eps) * _np(w)
        _close(n, ref_n, (H / 2 + 10) * U * np.abs(ref_n) * (1 + 2.0 ** -10) + _round(ref_n, dtype) * (1 + 2.0 ** -7), f"n of res {T}x{H}")


def test_small_eps_in_fp16():
    """fp16 rows of subnormal values whose squares are far above eps."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(7)
    eps = float(np.float32(1e-30))
    for H in (7, 300, 4096):
        res = torch.from_numpy(rng.standard_normal((4, H)) * 1e-6).half().cuda()
        _, n = moeq.block_norm(res, eps=eps)
        ref = _np(res) / norms.rms(_np(res), eps)
        _close(n, ref, (H / 2 + 10) * U * np.abs(ref) + _round(ref, F16) * (1 + 2.0 ** -7), H)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_infinities_and_nan_beside_large_rows(dtype):
    """A row with an infinity or a NaN gives none of finite value where that
    stands, and leaves the rows beside it, large or not, as they are alone."""
    from bit_quantized_moe_token_amd import moeq
    for H in (40, 700, 4096):
        rng = np.random.default_rng(H)
        v = _rows(rng, 6, H, 1e20, dtype)
        v[0] = torch.from_numpy(rng.standard_normal(H)).to(dtype)
        v[3, 5], v[4, 0] = float("inf"), float("nan")
        _, n = moeq.block_norm(v)
        assert bool(torch.isnan(n[3, 5])) and bool(torch.isnan(n[4]).all())
        assert not n[3, :5].any() and not n[3, 6:].any()
        for i in (0, 1, 2, 5):
            assert bool(torch.isfinite(n[i]).all())
            assert torch.equal(n[i], moeq.block_norm(v[i:i + 1].contiguous())[1][0])


def _grad_tol(q, r, d_r, d_n, alpha, eps, T, H):
    """Bounds on the fp32 error of every gradient before its last rounding, as
    in the norms' own tests; their counts, of eight roundings and more, grow
    by at most two here: a quarter."""
    u = 1.25 * U
    a, b = 1 / norms.rms(r, eps), 1 / norms.rms(q["y"], eps)
    g, un, v = np.abs(d_n * q["w_pre"]), np.abs(r * a), np.abs(q["y"]) * b
    gate, wp = np.abs(q["gate"]), np.abs(q["w_post"])
    mag = np.abs(d_r) + a * (g + un * np.mean(g * un, axis=1, keepdims=True))
    e_dr = (2 * H + 16) * u * mag
    cols = lambda mags, errs: errs.sum(0) + T * u * mags.sum(0)
    tol = {"d_residual": abs(alpha) * (e_dr + 2 * u * mag)}
    tol["d_w_pre"] = cols(np.abs(d_n) * un, (H / 2 + 8) * u * np.abs(d_n) * un)
    c, e_c = mag * gate * wp, e_dr * gate * wp
    m = np.mean(c * v, axis=1, keepdims=True)
    tol["d_y"] = b * (e_c + v * (np.mean(e_c * v, axis=1, keepdims=True) + (2 * H + 16) * u * m) + (H + 16) * u * (c + v * m))
    tol["d_w_post"] = cols(mag * gate * v, (e_dr + (H / 2 + 8) * u * mag) * gate * v)
    d, e = mag * v * wp, (e_dr + (H / 2 + 8) * u * mag) * v * wp
    tol["d_gate"] = e if q["gate"].ndim == 2 else cols(d, e)
    return tol


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("m", range(len(MAGNITUDES)))
def test_gradients_of_any_magnitude(m, types):
    from bit_quantized_moe_token_amd import moeq
    dtype, res_dtype = types
    my, mr, eps = MAGNITUDES[m]
    eps = float(np.float32(eps))
    down = 1e-15 if eps < 1e-37 else 1.0          # (1 / rms^2 is about 1e40 there)
    for H in WIDTHS:
        rng = np.random.default_rng(5000 + 1000 * m + H)
        T = 3 if H > 1 else 1
        v = dict(y=_rows(rng, T, H, my, dtype), r=_rows(rng, T, H, mr, res_dtype))
        one = lambda *s: torch.from_numpy(1 + 0.2 * rng.standard_normal(s)).to(dtype).cuda()
        v.update(w_pre=one(H), w_post=one(H), gate=one(H) if m % 2 else one(T, H))
        d_n = torch.from_numpy(rng.standard_normal((T, H)) * down).to(dtype).cuda()
        d_r = torch.from_numpy(rng.standard_normal((T, H)) * down).to(res_dtype).cuda() if m % 3 else None
        got = moeq.block_norm_grad(v["r"], d_n, v["y"], d_res=d_r, w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"],
                                   alpha=0.75, eps=eps)
        q = {k: _np(t) for k, t in v.items()}
        dr = _np(d_r) if d_r is not None else np.zeros((T, H))
        ref = norms.block_norm_grad(q["r"], q["y"], dr, _np(d_n), q["w_pre"], q["w_post"], q["gate"], 0.75, eps, True)
        tol = _grad_tol(q, q["r"], dr, _np(d_n), 0.75, eps, T, H)
        assert set(got) == set(ref)
        for k in ref:
            _close(got[k], ref[k], tol[k] * (1 + 2.0 ** -8) + _round(ref[k], got[k].dtype) * (1 + 2.0 ** -6), f"{k} {T}x{H}")


def test_large_gradients_of_small_rows():
    """Rows of order 1 whose incoming gradients, summed against them, leave
    fp32: d_n of 1e36 and r' of 1e10."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(3)
    for H in (64, 4096):
        r = torch.from_numpy(rng.standard_normal((3, H)) * 1e10).float().cuda()
        d_n = torch.from_numpy(rng.standard_normal((3, H)) * 1e36).float().cuda()
        got = moeq.block_norm_grad(r, d_n)["d_residual"]
        ref = norms.block_norm_grad(_np(r), None, np.zeros((3, H)), _np(d_n), None, None, None, 1.0, 1e-6, True)["d_residual"]
        a = 1 / norms.rms(_np(r), 1e-6)
        g, u = np.abs(_np(d_n)), np.abs(_np(r) * a)
        mag = a * (g + u * np.mean(g * u, axis=1, keepdims=True))
        _close(got, ref, 1.25 * (2 * H + 16) * U * mag + _round(ref, F32), H)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(1, 64, 40), (5, 4096, 33), (40, 200, 130)])
def test_linear_i8_of_large_rows(T, K, N, dtype):
    """Rows up to the type's largest values with channel scales that bring the
    result back: three fp32 roundings, then one to the output's type."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(K)
    x = rng.uniform(-1, 1, (T, K)) * np.exp2(rng.choice([0, 60, 100, 127], (T, 1)))
    x = torch.from_numpy(x).to(dtype).cuda()
    wq = torch.from_numpy(rng.integers(-127, 128, (N, K)).astype(np.int8)).cuda()
    sw = torch.from_numpy((rng.uniform(0.5, 1.5, N) * 2.0 ** rng.choice([-120, -60, -20], N)).astype(np.float32)).cuda()
    xq, sx = moeq.quantize_i8(x)
    ints = xq.cpu().numpy().astype(np.float64) @ wq.cpu().numpy().astype(np.float64).T
    ref = ints * sx.cpu().numpy().astype(np.float64)[:, None] * sw.cpu().numpy().astype(np.float64)
    assert np.abs(ref).max() < 2.0 ** 126
    for y in (moeq.linear_i8(x, wq, sw), moeq.gemm_i8(xq, sx, wq, sw, out_dtype=dtype)):
        _close(y, ref, 3 * U * np.abs(ref) * (1 + 2.0 ** -8) + _round(ref, dtype) * (1 + 2.0 ** -8), (T, K, N))


def test_gemm_i8_with_scales_at_the_ends_of_fp32():
    from bit_quantized_moe_token_amd import moeq
    xq = torch.full((6, 1000), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((3, 1000), -127, dtype=torch.int8, device="cuda")
    sx = torch.tensor([3e38, -3e38, 2.0 ** 95, float("inf"), float("nan"), 1.0], device="cuda")
    sw = torch.tensor([2.0 ** -120, 2.0 ** -149, 1.0], device="cuda")
    y = _np(moeq.gemm_i8(xq, sx, wq, sw, out_dtype=F32))
    ref = -16129000.0 * _np(sx)[:, None] * _np(sw)
    large = np.abs(ref) > 3.4028235e38
    assert np.array_equal(np.isnan(y), np.isnan(ref)) and np.array_equal(np.isinf(y), large & ~np.isnan(ref))
    ok = ~np.isnan(ref) & ~large
    assert np.all(np.abs(y - ref)[ok] <= 3 * U * np.abs(ref[ok]) + 4 * 2.0 ** -150)


@pytest.mark.parametrize("H", [40, 700, 4096, 8192, 10000])
def test_gradient_of_a_block_without_post_norm_does_not_read_it(H):
    """d_y = dr gate, whatever y holds, where y is not normed; d_gate is dr y."""
    from bit_quantized_moe_token_amd import moeq
    g = torch.Generator(device="cuda").manual_seed(H)
    r, y, d_n, gate = (torch.randn(s, generator=g, device="cuda") for s in ((3, H), (3, H), (3, H), (H,)))
    kw = dict(gate=gate, post_norm=False, alpha=0.5)
    want = moeq.block_norm_grad(r, d_n, y, **kw)
    bad = y.clone()
    bad[1, 3], bad[1, 7], bad[2, H - 1] = float("inf"), float("-inf"), float("nan")
    got = moeq.block_norm_grad(r, d_n, bad, **kw)
    assert torch.equal(got["d_y"], want["d_y"]) and torch.equal(got["d_residual"], want["d_residual"])
    same = torch.ones(H, dtype=torch.bool)
    same[[3, 7, H - 1]] = False
    assert torch.equal(got["d_gate"][same.cuda()], want["d_gate"][same.cuda()])
    assert not torch.isfinite(got["d_gate"][~same.cuda()]).any()
