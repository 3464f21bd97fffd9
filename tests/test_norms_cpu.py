"""Refusals of the norm entry points (on the host, nothing is enqueued), and
the fp64 gradients against differences."""

import ctypes

import numpy as np
import pytest

from oracle import norms

P = 4096


@pytest.fixture(scope="module")
def L():
    from bit_quantized_moe_token_amd import _lib
    return _lib.lib()


def _d(T=4, H=64, dtype=0, res=0, w_pre=P, w_post=P, gate=P, per_token=0, post=1, alpha=1.0, eps=1e-6):
    from bit_quantized_moe_token_amd import _lib
    return ctypes.byref(_lib.Norm(T, H, dtype, res, w_pre, w_post, gate, per_token, post, alpha, eps))


BAD = [(dict(T=-1), 1), (dict(T=1 << 22), 2), (dict(H=0), 1), (dict(H=32769), 2), (dict(dtype=3), 1), (dict(res=2), 1),
       (dict(dtype=1, res=0), 1), (dict(post=2), 1), (dict(post=0), 1), (dict(per_token=2), 1), (dict(eps=0.0), 1),
       (dict(eps=float("nan")), 1), (dict(alpha=float("inf")), 1), (dict(w_pre=4097), 1), (dict(gate=4097), 1),
       (dict(dtype=1, res=1, w_post=4098), 1)]


@pytest.mark.parametrize("bad,status", BAD, ids=lambda v: str(v))
def test_descriptions_refused(L, bad, status):
    assert L.moeq_block_norm(_d(**bad), P, P, P, P, None) == status
    assert L.moeq_block_norm_grad(_d(**bad), P, P, P, P, P, P, P, P, P, P, 1 << 24, None) == status
    assert L.moeq_last_error()


def test_operands_refused(L):
    assert L.moeq_block_norm(None, P, P, P, P, None) == 1
    for a in ((None, P, P, P), (P, P, None, P), (P, P, P, None), (4097, P, P, P), (P, 4097, P, P), (P, P, P, 4097)):
        assert L.moeq_block_norm(_d(), *a, None) == 1, a
    # without a block there is nothing to gate or to norm after it
    assert L.moeq_block_norm(_d(w_post=None), P, None, P, P, None) == 1
    assert L.moeq_block_norm(_d(gate=None), P, None, P, P, None) == 1
    # no tokens: matrices may be null
    assert L.moeq_block_norm(_d(T=0), None, None, None, None, None) == 0
    n = ctypes.c_size_t(0)
    assert L.moeq_block_norm_grad_workspace_size(4, 64, ctypes.byref(n)) == 0 and n.value >= 3 * 64 * 4
    size = n.value
    good = dict(res=P, y=P, d_res=P, d_n=P, d_r=P, d_y=P, wp=P, wq=P, dg=P, ws=P, n=size)
    for bad, status in ((dict(res=None), 1), (dict(d_n=None), 1), (dict(d_r=None), 1), (dict(d_y=None), 1),
                        (dict(dg=None), 1), (dict(ws=None), 1), (dict(ws=4104), 1), (dict(n=size - 1), 3),
                        (dict(wp=4098), 1), (dict(d_res=4097), 1), (dict(dg=4098), 1)):
        a = dict(good, **bad)
        assert L.moeq_block_norm_grad(_d(), a["res"], a["y"], a["d_res"], a["d_n"], a["d_r"], a["d_y"], a["wp"], a["wq"],
                                      a["dg"], a["ws"], a["n"], None) == status, bad
    assert L.moeq_block_norm_grad(_d(gate=None), P, P, P, P, P, P, P, P, P, P, size, None) == 1    # d_gate without gate
    assert L.moeq_block_norm_grad(_d(post=0, w_post=None), P, P, P, P, P, P, P, P, P, P, size, None) == 1
    assert L.moeq_block_norm_grad_workspace_size(1, 32769, ctypes.byref(n)) == 2


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "vector", "token"])
@pytest.mark.parametrize("block", [True, False])
def test_oracle_gradients_against_differences(block, gate, post):
    rng = np.random.default_rng(5)
    T, H, alpha, eps = 3, 7, 0.6, 1e-3
    if not block and gate != "none":
        pytest.skip("no gate without a block")
    v = dict(res=rng.standard_normal((T, H)), w_pre=rng.standard_normal(H))
    if block:
        v["y"] = rng.standard_normal((T, H))
        if post:
            v["w_post"] = rng.standard_normal(H)
        if gate != "none":
            v["gate"] = rng.standard_normal(H if gate == "vector" else (T, H))
    c1, c2 = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    get = lambda q, k: q.get(k)

    def loss(q):
        r, n = norms.block_norm(q["res"], get(q, "y"), q["w_pre"], get(q, "w_post"), get(q, "gate"), alpha, eps, post)
        return float((c1 * r + c2 * n).sum())

    r, _ = norms.block_norm(v["res"], get(v, "y"), v["w_pre"], get(v, "w_post"), get(v, "gate"), alpha, eps, post)
    g = norms.block_norm_grad(r, get(v, "y"), c1, c2, v["w_pre"], get(v, "w_post"), get(v, "gate"), alpha, eps, post)
    names = dict(res="d_residual", y="d_y", w_pre="d_w_pre", w_post="d_w_post", gate="d_gate")
    assert {names[k] for k in v} == set(g)
    h = 1e-5
    for k in v:
        num = np.zeros_like(v[k])
        for i in np.ndindex(v[k].shape):
            up, dn = {a: b.copy() for a, b in v.items()}, {a: b.copy() for a, b in v.items()}
            up[k][i] += h
            dn[k][i] -= h
            num[i] = (loss(up) - loss(dn)) / (2 * h)
        # central differences: h^2 times a third derivative of at most some hundreds here
        assert np.allclose(num, g[names[k]], rtol=1e-6, atol=1e-6), k
