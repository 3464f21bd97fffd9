"""Refusals of scored routing, the combine of expert-sorted rows and the
adapters (on the host, nothing is enqueued), and their fp64 forms against
closed forms, differences and brute force."""

import ctypes
import itertools
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from bit_quantized_moe_token_amd import build
from oracle import products, requests, scores

P = 4096


@pytest.fixture(scope="module")
def L():
    from bit_quantized_moe_token_amd import _lib
    return _lib.lib()


def _scoring(score=0, renorm=1, scale=1.0, bias=P, groups=4, top=2, group_score=1):
    from bit_quantized_moe_token_amd import _lib
    return ctypes.byref(_lib.Scoring(score, renorm, scale, bias, groups, top, group_score))


def _routing(**none):
    from bit_quantized_moe_token_amd import _lib
    names = ("topk_ids", "topk_gates", "expert_offsets", "sorted_pairs", "pair_pos")
    return ctypes.byref(_lib.Routing(*[none.get(n, P) for n in names]))


def _route(L, d=None, logits=P, ld=64, dt=1, T=20, E=64, k=6, out=None, ws=None, n=0):
    return L.moeq_route_scored(d or _scoring(), logits, ld, dt, T, E, k, out or _routing(), ws, n, None)


def _grad(L, d=None, logits=P, ld=64, dt=1, T=20, E=64, k=6, ids=P, dg=P, out=P, ldd=64):
    return L.moeq_route_scored_grad(d or _scoring(), logits, ld, dt, T, E, k, ids, dg, out, ldd, None)


@pytest.mark.parametrize("bad", [dict(score=2), dict(score=-1), dict(renorm=2), dict(scale=float("inf")),
                                 dict(scale=float("nan"))], ids=str)
def test_scoring_refused_by_both(L, bad):
    assert _route(L, _scoring(**bad)) == 1 and L.moeq_last_error()
    assert _grad(L, _scoring(**bad)) == 1


@pytest.mark.parametrize("bad", [dict(groups=0), dict(groups=-1), dict(groups=5), dict(groups=128), dict(top=0), dict(top=5),
                                 dict(groups=16, top=1), dict(group_score=2), dict(groups=64, top=64), dict(bias=4098)],
                         ids=str)
def test_groups_refused(L, bad):
    assert _route(L, _scoring(**bad)) == 1 and L.moeq_last_error()


def test_group_choice_is_not_looked_at_with_one_group(L):
    assert _route(L, _scoring(groups=1, top=1, group_score=7), T=4097) == 3      # (the check that comes last)


@pytest.mark.parametrize("bad,status", [
    (dict(logits=None), 1), (dict(logits=4098), 1), (dict(ld=63), 1), (dict(dt=3), 1), (dict(T=-1), 1), (dict(E=0), 1),
    (dict(E=257, ld=300), 1), (dict(k=0), 1), (dict(k=65), 1), (dict(T=1 << 22), 2), (dict(T=4000000, E=256, ld=256, k=200), 2)])
def test_routing_operands_refused(L, bad, status):
    one = _scoring(groups=1, top=1)
    assert _route(L, one, **bad) == status and L.moeq_last_error()
    assert _grad(L, one, **bad) == status


def test_routing_outputs_refused(L):
    for n in ("topk_ids", "topk_gates", "expert_offsets", "sorted_pairs", "pair_pos"):
        assert _route(L, out=_routing(**{n: None})) == 1, n
    assert L.moeq_route_scored(None, P, 64, 1, 4, 64, 6, _routing(), None, 0, None) == 1
    assert L.moeq_route_scored(_scoring(), P, 64, 1, 4, 64, 6, None, None, 0, None) == 1
    assert _route(L, T=4097) == 3 and _route(L, T=4097, ws=P, n=100) == 3
    for bad in (dict(ids=None), dict(dg=None), dict(ids=4097), dict(dg=4098), dict(out=None), dict(ldd=63), dict(out=4098)):
        assert _grad(L, **bad) == 1, bad
    assert _grad(L, T=0, logits=None, ids=None, dg=None, out=None) == 0
    assert L.moeq_route_scored_grad(None, P, 64, 1, 4, 64, 6, P, P, P, 64, None) == 1


def _combine(L, rows=P, ldr=32, Pn=8, dt=0, pos=P, gates=P, T=4, k=2, N=32, base=P, ldb=32, out=P, ldo=32, odt=0):
    return L.moeq_combine(rows, ldr, Pn, dt, pos, gates, T, k, N, base, ldb, out, ldo, odt, None)


def _cgrad(L, rows=P, ldr=32, Pn=8, dt=0, pos=P, gates=P, T=4, k=2, N=32, base=P, ldb=32, out=P, ldo=32, odt=0, dg=P):
    return L.moeq_combine_grad(base, ldb, odt, pos, gates, T, k, N, rows, ldr, Pn, dt, out, ldo, dg, None)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=None), 1), (dict(rows=4097), 1), (dict(ldr=31), 1), (dict(dt=3), 1), (dict(dt=0, odt=2), 1), (dict(odt=5), 1),
    (dict(dt=2, odt=0), 1), (dict(pos=None), 1), (dict(pos=4098), 1), (dict(gates=4098), 1), (dict(T=-1), 1), (dict(Pn=-1), 1),
    (dict(k=0), 1), (dict(k=257), 1), (dict(N=0), 1), (dict(N=(1 << 20) + 1), 2), (dict(T=1 << 22), 2),
    (dict(Pn=(1 << 29) + 1), 2), (dict(T=4000000, k=200), 2), (dict(base=4097), 1), (dict(ldb=31), 1), (dict(out=None), 1),
    (dict(ldo=31), 1), (dict(ldr=1 << 31), 2)])
def test_combine_refused(L, bad, status):
    assert _combine(L, **bad) == status and L.moeq_last_error()
    assert _cgrad(L, **bad) == status


def test_combine_without_work(L):
    assert _combine(L, T=0, rows=None, pos=None, gates=None, base=None, out=None) == 0
    assert _cgrad(L, T=0, rows=None, pos=None, base=None, out=None) == 0
    assert _cgrad(L, gates=None) == 1            # d_gates without gates
    assert _cgrad(L, dg=4098) == 1 and _cgrad(L, base=None) == 1


def _adapters(L, a=P, lda=64, sa=64 * 256, b=P, ldb=256, sb=256 * 32, scale=P, ranks=P, n=3, R=256, N=32, K=64, dt=0, x=P, ldx=64,
              ids=P, T=4, y=P, ldy=32, out=P, ldo=32, ydt=0, ws=P, size=1 << 20):
    from bit_quantized_moe_token_amd import _lib
    s = _lib.AdaptersSet(a, b, lda, sa, ldb, sb, scale, ranks, n, R, N, K, dt)
    return L.moeq_adapters(ctypes.byref(s), x, ldx, ids, T, y, ldy, out, ldo, ydt, ws, size, None)


@pytest.mark.parametrize("bad,status", [
    (dict(a=None), 1), (dict(a=4097), 1), (dict(lda=63), 1), (dict(sa=-1), 1), (dict(b=None), 1), (dict(b=4097), 1),
    (dict(ldb=255), 1), (dict(sb=-1), 1), (dict(scale=4098), 1), (dict(ranks=4098), 1), (dict(n=0), 1),
    (dict(n=(1 << 20) + 1), 2), (dict(R=0), 1), (dict(R=257, ldb=257), 2), (dict(N=0), 1), (dict(N=(1 << 20) + 1), 2),
    (dict(K=0), 1), (dict(K=(1 << 20) + 1), 2), (dict(dt=1), 1), (dict(ydt=2), 1), (dict(x=None), 1), (dict(ldx=63), 1),
    (dict(ids=None), 1), (dict(ids=4097), 1), (dict(T=-1), 1), (dict(T=1 << 22), 2), (dict(y=None), 1), (dict(ldy=31), 1),
    (dict(out=None), 1), (dict(ldo=31), 1), (dict(ydt=1, y=4098), 1), (dict(ws=None), 1), (dict(ws=4104), 1),
    (dict(size=0), 3)])
def test_adapters_refused(L, bad, status):
    assert _adapters(L, **bad) == status and L.moeq_last_error()


def test_adapters_sizes(L):
    n = ctypes.c_size_t(0)
    assert L.moeq_adapters(None, P, 64, P, 4, P, 32, P, 32, 0, P, 1 << 20, None) == 1
    assert _adapters(L, T=0, x=None, ids=None, y=None, out=None, ws=None, size=0) == 0
    assert L.moeq_adapters_workspace_size(4, 256, 64, ctypes.byref(n)) == 0 and n.value >= 4 * 256 * 4
    assert _adapters(L, size=n.value - 1) == 3
    for bad, status in (((-1, 8, 64), 1), ((4, 0, 64), 1), ((4, 257, 64), 2), ((4, 8, 0), 1), ((1 << 22, 8, 64), 2)):
        assert L.moeq_adapters_workspace_size(*bad, ctypes.byref(n)) == status
    assert L.moeq_adapters_workspace_size(4, 8, 64, None) == 1


def test_sizes_beyond_32_bits_are_refused():
    from bit_quantized_moe_token_amd import moeq
    for bad in ((2 ** 32 + 4, 8, 64), (4, 2 ** 32 + 8, 64), (4, 8, 2 ** 32 + 64)):
        with pytest.raises(ValueError):
            moeq.adapters_workspace_size(*bad)


@pytest.mark.parametrize("T", [5, 0, 5000])
def test_tensors_of_a_routing_stand_alone(T):
    """Each output has its own memory, so that keeping one keeps no other, and
    its own version counter; the workspace is a tensor also where none is needed."""
    import torch
    from bit_quantized_moe_token_amd import moeq
    r = moeq.RoutingOut(T, 8, 2, "cpu")
    all_of = {n: getattr(r, n) for n in ("ids", "gates", "offsets", "sorted_pairs", "pair_pos")}
    assert [tuple(t.shape) for t in all_of.values()] == [(T, 2), (T, 2), (9,), (2 * T,), (2 * T,)]
    for n, t in all_of.items():
        assert t.untyped_storage().nbytes() == 4 * t.numel() and not t._is_view(), n
        before = {m: o._version for m, o in all_of.items()}
        moeq._written(t)
        assert [m for m, o in all_of.items() if o._version != before[m]] == [n]
    assert r.ws.dtype == torch.uint8 and r.ws.numel() == max(1, r.ws_bytes) and r.ws is r.ws


# ---- the fp64 forms

def test_scores_closed_forms():
    assert np.allclose(scores.scores(np.zeros(5), "softmax"), 0.2)
    assert np.allclose(scores.scores(np.log([1.0, 3.0]), "softmax"), [0.25, 0.75])
    assert np.allclose(scores.scores(np.array([0.0, np.log(3.0), -np.log(3.0)]), "sigmoid"), [0.5, 0.75, 0.25])
    ninf = -np.inf
    assert (scores.scores(np.array([ninf, ninf]), "softmax") == 0).all()
    assert (scores.scores(np.array([ninf, np.nan]), "sigmoid") == 0).all()
    assert (scores.scores(np.array([np.inf, 1.0, np.inf]), "softmax") == [0.5, 0, 0.5]).all()
    # all out: the lowest ids, gates zero
    ids, g = scores.route(np.full((1, 6), ninf), 3)
    assert ids.tolist() == [[0, 1, 2]] and (g == 0).all()


@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_choice_by_brute_force(group_score):
    """Over all subsets: the chosen ones have the largest sum of choices
    within the groups whose worth is largest."""
    rng = np.random.default_rng(3)
    for _ in range(20):
        l, bias = rng.standard_normal(12), 0.2 * rng.standard_normal(12)
        s = 1 / (1 + np.exp(-l))
        c = s + bias
        worth = [sum(sorted(c[g * 3:g * 3 + 3])[-(1 if group_score == "max" else 2):]) for g in range(4)]
        kept = max(itertools.combinations(range(4), 2), key=lambda p: sum(worth[g] for g in p))
        inside = [e for e in range(12) if e // 3 in kept]
        want = max(itertools.combinations(inside, 4), key=lambda p: sum(c[e] for e in p))
        got = scores.choose(l, 4, "sigmoid", bias, 4, 2, group_score)
        assert sorted(got) == sorted(want) and (np.diff(c[got]) <= 0).all()


def test_ties_go_to_the_lowest():
    assert scores.choose(np.zeros(8), 3, "softmax", None, 1, 1, "max") == [0, 1, 2]
    assert scores.choose(np.zeros(8), 3, "sigmoid", np.zeros(8), 4, 2, "top2") == [0, 1, 2]
    assert scores.choose(np.array([0.0, 1, 1, 0]), 2, "softmax", None, 2, 2, "max") == [1, 2]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    T, E, k, scale, h = 3, 7, 3, 1.7, 1e-5
    l, dg = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    got, mag = scores.route_grad(l, ids, dg, score, renorm, scale)
    assert (np.abs(got) <= mag + 1e-15).all()
    f = lambda v, t: (scores.gates(v, ids[t], score, renorm, scale) * dg[t]).sum()
    for t in range(T):
        for e in range(E):
            up, dn = l[t].copy(), l[t].copy()
            up[e] += h
            dn[e] -= h
            # central differences: h^2 times a third derivative of a few units
            assert abs((f(up, t) - f(dn, t)) / (2 * h) - got[t, e]) < 1e-8


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_gradient_without_cancellation(score, renorm):
    """On ordinary rows the same as route_grad; of a row that one expert leads
    by far, what the closed forms give."""
    rng = np.random.default_rng(5)
    T, E, k = 4, 9, 4
    l, dg = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    a, mag = scores.route_grad_apart(l, ids, dg, score, renorm, -1.5)
    assert np.allclose(a, scores.route_grad(l, ids, dg, score, renorm, -1.5)[0], rtol=1e-12, atol=1e-14)
    assert (np.abs(a) <= mag * (1 + 1e-12)).all()
    for lead in (5.0, 20.0, 60.0):
        q = np.exp(-lead)
        if score == "softmax" and not renorm:      # s (1 - s), and -s / 8 of it for each of the others
            a, _ = scores.route_grad_apart([[lead] + [0.0] * 8], [[0]], [[1.0]], score, renorm)
            rest = 8 * q / (1 + 8 * q)
            assert np.allclose(a[0], [rest / (1 + 8 * q)] + [-rest / 8 / (1 + 8 * q)] * 8, rtol=1e-13, atol=0)
        elif score == "softmax":                   # two experts: s_0 s_1 (dg_0 - dg_1)
            a, _ = scores.route_grad_apart([[lead, 0.0, 3.0]], [[0, 1]], [[2.0, -1.0]], score, renorm)
            assert np.allclose(a[0], [3 * q / (1 + q) ** 2, -3 * q / (1 + q) ** 2, 0], rtol=1e-13, atol=0)


def test_combine_and_its_gradient():
    rng = np.random.default_rng(2)
    T, k, N = 3, 2, 5
    rows, dy, gates = rng.standard_normal((6, N)), rng.standard_normal((T, N)), rng.standard_normal((T, k))
    pos = rng.permutation(6)
    pos[3] = -1
    y, _ = products.combine(rows, pos, gates, None, T, k)
    d_rows, d_gates, _ = products.combine_grad(dy, pos, gates, rows, 6, np.zeros((6, N)))
    # linear in the rows and in the gates: <dy, y> is the product of either with its gradient
    assert np.isclose((d_rows * rows).sum(), (dy * y).sum())
    assert np.isclose((d_gates * gates).sum(), (dy * y).sum())
    assert d_gates[1, 1] == 0
    ones, _ = products.combine(rows, np.arange(6), None, np.ones((T, N)), T, k)
    assert np.allclose(ones, 1 + rows.reshape(T, k, N).sum(1))


def test_adapters_as_dense_matrices():
    rng = np.random.default_rng(4)
    x, a, b, y = (rng.standard_normal(s) for s in ((5, 6), (3, 4, 6), (3, 7, 4), (5, 7)))
    ids, scale, ranks = [2, -1, 0, 2, 3], np.array([0.5, 1.0, 2.0]), [2, 4, 9]
    out, _, _ = requests.adapters(x, a, b, ids, y, scale, ranks)
    assert np.allclose(out[[1, 4]], y[[1, 4]])
    assert np.allclose(out[0], y[0] + 2 * (b[2] @ a[2]) @ x[0])
    assert np.allclose(out[2], y[2] + 0.5 * (b[0][:, :2] @ a[0][:2]) @ x[2])


def test_adapters_adapter_by_adapter():
    rng = np.random.default_rng(6)
    x, a, b, y = (rng.standard_normal(s) for s in ((40, 6), (3, 4, 6), (3, 7, 4), (40, 7)))
    ids, scale, ranks = rng.integers(-1, 4, 40), np.array([0.5, -1.0, 2.0]), [2, 0, 9]
    for kw in ({}, dict(scale=scale), dict(scale=scale, ranks=ranks)):
        for p, q in zip(requests.adapters(x, a, b, ids, y, **kw), requests.adapters_of_many_rows(x, a, b, ids, y, **kw)):
            assert np.allclose(p, q, rtol=1e-13, atol=1e-13)


@pytest.mark.skipif(not os.path.exists(build.HIPCC) and not shutil.which(build.HIPCC), reason="no compiler")
@pytest.mark.parametrize("name,kernels", [("score", 9), ("combine", 9), ("adapters", 20)])
def test_kernels_use_no_scratch(name, kernels):
    """Choices, rows and MFMA operands are held in registers: the compiler
    reports no scratch for any kernel."""
    src = os.path.join(build.CSRC, name + ".hip")
    r = subprocess.run([build.HIPCC, *build.CFLAGS, "-Rpass-analysis=kernel-resource-usage", "-S", "--cuda-device-only", src,
                        "-o", os.devnull], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", r.stderr, re.S)
    assert len(found) >= kernels
    assert not [n for n, size in found if int(size)]
