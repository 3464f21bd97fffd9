"""Refusals of the product entry points (checked on the host, nothing is
enqueued), and the fp64 forms against differences and closed forms."""

import ctypes

import numpy as np
import pytest

from oracle import products


@pytest.fixture(scope="module")
def L():
    from bit_quantized_moe_token_amd import _lib
    return _lib.lib()


P16 = 4096


def _g(E=2, P=8, T=4, k=2, off=P16, pairs=P16):
    from bit_quantized_moe_token_amd import _lib
    return ctypes.byref(_lib.Groups(off, pairs, E, P, T, k))


def _gemm(L, g=None, x=P16, ldx=64, w=P16, ldw=64, sw=64 * 32, trans=0, N=32, K=64, dt=0, y=P16, ldy=32, ydt=0):
    return L.moeq_grouped_gemm(g or _g(), x, ldx, w, ldw, sw, trans, N, K, dt, y, ldy, ydt, None)


BAD_GROUPS = [dict(T=0), dict(E=0), dict(E=257), dict(P=-1), dict(T=-1), dict(k=0), dict(off=None), dict(pairs=None),
              dict(off=4098), dict(pairs=4097)]


@pytest.mark.parametrize("bad", BAD_GROUPS, ids=lambda b: "-".join(f"{k}={v}" for k, v in b.items()))
def test_groups_refused(L, bad):
    g = _g(**bad)
    p = P16
    assert _gemm(L, g) == 1
    assert L.moeq_grouped_wgrad(g, p, 32, p, 64, 32, 64, 0, p, 64, 2048, 1, None) == 1
    assert L.moeq_gemm_i8(g, p, 64, p, p, 64, 2048, p, 32, 64, p, 32, 0, None) == 1
    assert L.moeq_linear_i8(g, p, 64, 0, p, 64, 2048, p, 32, 64, p, 32, 0, p, 1 << 20, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(x=4097), 1), (dict(w=4097), 1), (dict(y=4097), 1),
    (dict(ldx=63), 1), (dict(ldw=63), 1), (dict(ldy=31), 1), (dict(trans=2), 1), (dict(trans=1, ldw=31), 1),
    (dict(N=0), 1), (dict(K=0), 1), (dict(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), 2), (dict(dt=1), 1),
    (dict(dt=3), 1), (dict(ydt=2), 1), (dict(sw=-1), 1), (dict(ldx=1 << 31), 2), (dict(ydt=1, y=4098), 1),
])
def test_grouped_gemm_refused(L, bad, status):
    assert _gemm(L, **bad) == status
    assert L.moeq_last_error()


def test_too_many_rows(L):
    p, n = P16, (1 << 29) + 1
    g = _g(P=n, T=n)
    assert _gemm(L, g) == 2 and L.moeq_grouped_wgrad(g, p, 32, p, 64, 32, 64, 0, p, 64, 2048, 1, None) == 2
    assert L.moeq_gemm_i8(g, p, 64, p, p, 64, 2048, p, 32, 64, p, 32, 0, None) == 2
    assert L.moeq_quantize_i8(p, 64, 1 << 22, 64, 0, p, 64, p, None) == 2


def test_null_groups(L):
    assert L.moeq_grouped_gemm(None, P16, 64, P16, 64, 0, 0, 32, 64, 0, P16, 32, 0, None) == 1


def test_no_rows_is_no_work(L):
    # nothing is read or written, whatever the pointers
    assert _gemm(L, _g(P=0, T=0), x=None, w=None, y=None) == 0
    assert L.moeq_gemm_i8(_g(P=0), None, 64, None, None, 64, 0, None, 32, 64, None, 32, 0, None) == 0
    assert L.moeq_linear_i8(_g(P=0), None, 64, 0, None, 64, 0, None, 32, 64, None, 32, 0, None, 0, None) == 0
    assert L.moeq_quantize_i8(None, 64, 0, 64, 0, None, 64, None, None) == 0


def test_wgrad_refused(L):
    def call(g=None, dy=P16, lddy=32, x=P16, ldx=64, N=32, K=64, dt=0, dw=P16, lddw=64, sd=2048, wdt=1):
        return L.moeq_grouped_wgrad(g or _g(), dy, lddy, x, ldx, N, K, dt, dw, lddw, sd, wdt, None)
    for bad in (dict(dy=None), dict(x=None), dict(dw=None), dict(lddy=31), dict(ldx=63), dict(lddw=63), dict(sd=2047),
                dict(dt=1), dict(wdt=2), dict(dw=4098), dict(N=0), dict(K=-1)):
        assert call(**bad) == 1, bad
    assert call(N=(1 << 20) + 1, lddy=1 << 21, sd=1 << 40) == 2


def test_i8_refused(L):
    def call(g=None, x=P16, ldx=64, sx=P16, w=P16, ldw=64, sw=P16, N=32, K=64, y=P16, ldy=32, ydt=0):
        return L.moeq_gemm_i8(g or _g(), x, ldx, sx, w, ldw, 2048, sw, N, K, y, ldy, ydt, None)
    for bad in (dict(x=None), dict(sx=None), dict(w=None), dict(sw=None), dict(y=None), dict(ldx=63), dict(ldw=63),
                dict(ldy=31), dict(ydt=3), dict(sx=4098), dict(sw=4097), dict(N=0), dict(K=0)):
        assert call(**bad) == 1, bad
    assert call(K=131072, ldx=1 << 18, ldw=1 << 18) == 2       # the sum could pass 32 bits
    p = P16
    n = ctypes.c_size_t(0)
    assert L.moeq_linear_i8_workspace_size(4, 65, ctypes.byref(n)) == 0 and n.value == 4 * (128 + 4)
    assert L.moeq_linear_i8_workspace_size(-1, 65, ctypes.byref(n)) == 1
    assert L.moeq_linear_i8_workspace_size(1, 131072, ctypes.byref(n)) == 2

    def lin(ws=p, n=4 * (128 + 4), dt=0):
        return L.moeq_linear_i8(_g(), p, 65, dt, p, 65, 4096, p, 32, 65, p, 32, 0, ws, n, None)
    assert lin(n=4 * 132 - 1) == 3
    assert lin(ws=None) == 1 and lin(ws=4104) == 1 and lin(dt=5) == 1
    for bad in (dict(x=None), dict(ldx=63), dict(rows=-1), dict(cols=0), dict(dt=4), dict(q=None), dict(s=None),
                dict(ldc=63)):
        a = dict(x=p, ldx=64, rows=4, cols=64, dt=0, q=p, ldc=64, s=p)
        a.update(bad)
        assert L.moeq_quantize_i8(a["x"], a["ldx"], a["rows"], a["cols"], a["dt"], a["q"], a["ldc"], a["s"], None) == 1, bad


def test_oracle_gradients_against_differences():
    """The loss sum(c * y): its differences in x and w equal the row gradient
    (scattered back to the source rows) and the matrix gradient."""
    rng = np.random.default_rng(0)
    T, K, N, k, off = 5, 6, 4, 2, np.array([0, 3, 3, 9])
    x, w, pairs = rng.standard_normal((T, K)), rng.standard_normal((3, N, K)), rng.integers(0, T * k, 10)
    c = rng.standard_normal((10, N))
    c[9] = 0
    src = products.source_rows(10, T, pairs, k)
    loss = lambda x, w: float((c * products.grouped(x, w, off, src, np.zeros((10, N)))).sum())
    drow = products.grouped(c, w.swapaxes(1, 2), off, np.arange(10), np.zeros((10, K)))
    dx = np.zeros((T, K))
    np.add.at(dx, src, drow)
    dw = products.wgrad(c, x, off, src)
    h = 1e-5
    for a, grad, f in ((x, dx, lambda v: loss(v, w)), (w, dw, lambda v: loss(x, v))):
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += h
            dn[i] -= h
            num[i] = (f(up) - f(dn)) / (2 * h)
        # the loss is linear in either operand: only the fp64 rounding of the difference is left
        assert np.allclose(num, grad, rtol=0, atol=1e-8)


def test_oracle_codes():
    q, s = products.code_i8(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1, np.nan, 0, 0], [2.0 ** -120] * 4],
                                     dtype=np.float32))
    assert q.tolist() == [[127, -64, 0, 2], [0] * 4, [0] * 4, [0] * 4]
    assert s[0] == 1 and s[1] == 1 and np.isnan(s[2]) and s[3] == 1


def test_host_tensors_refused():
    """Tensors in host memory never reach the library."""
    torch = pytest.importorskip("torch")
    from bit_quantized_moe_token_amd import moeq
    x, w, off = torch.zeros(4, 8).half(), torch.zeros(2, 6, 8).half(), torch.zeros(3).int()
    v = torch.zeros(8).half()
    for call in (lambda: moeq.grouped_gemm(x, w, off), lambda: moeq.grouped_wgrad(x, x, off), lambda: moeq.quantize_i8(x),
                 lambda: moeq.linear_i8(x, w[0].char(), torch.ones(6)), lambda: moeq.gemm_i8(x.char(), torch.ones(4), w[0].char(), torch.ones(6)),
                 lambda: moeq.block_norm(x, x, w_pre=v), lambda: moeq.block_norm_grad(x, x, x, w_pre=v),
                 lambda: moeq.grouped_gemm(None, w, off), lambda: moeq.block_norm(None), lambda: moeq.block_norm_grad(x, None)):
        with pytest.raises(TypeError):
            call()
