"""Scored routing and its gradient against the fp64 forms.

The chosen experts are compared exactly: choices are formed in 64 bits (or are
the logits' own order), and inputs here hold no two choices closer than that
but equal ones, which go to the lowest id.  Gates: formed in 64 bits from the
chosen logits and rounded once (half a step, 2^-24); a softmax over all E
divides by an fp32 sum of E exponentials, each within 2 steps (2^-22), in a
tree of at most 4 + 6 additions: 16 * 2^-24 in all.
"""

import numpy as np
import pytest

from oracle import scores

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


def _logits(T, E, dtype=F32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn((T, E), generator=g) + torch.randn((E,), generator=g)).to(dtype)


def _bias(E, seed=1):
    g = torch.Generator().manual_seed(seed)
    return 0.001 * (50 * torch.randn((E,), generator=g)).round()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(logits, k, score, bias, groups, top, group_score, renorm, scale, out=None, strided=False):
    from bit_quantized_moe_token_amd import moeq
    T, E = logits.shape
    dev = logits.cuda()
    if strided:
        wide = torch.full((T, E + 3), 7.0, dtype=logits.dtype, device="cuda")
        wide[:, 1:E + 1] = dev
        dev = wide[:, 1:E + 1]
    r = moeq.route_scored(dev, k, score=score, bias=bias.cuda() if bias is not None else None, groups=groups,
                          top_groups=top, group_score=group_score, renorm=renorm, scale=scale, out=out)
    ids, gates = scores.route(_np(logits), k, score, None if bias is None else _np(bias), groups, top, group_score, renorm,
                              scale)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    off, order, pos = scores.sort_pairs(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.sorted_pairs.cpu().numpy(), order) and np.array_equal(r.pair_pos.cpu().numpy(), pos)
    got = _np(r.gates)
    n = 16 if score == "softmax" and not renorm else 1.01
    bad = np.abs(got - gates) > n * 2.0 ** -24 * np.abs(gates) + 2.0 ** -149
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - gates).max()))
    return r


SHAPES = [(1, 1, 1, 1, 1), (1, 64, 6, 1, 1), (3, 5, 5, 1, 1), (16, 128, 8, 1, 1), (17, 128, 8, 1, 1), (16, 256, 8, 8, 4),
          (300, 256, 8, 8, 4), (64, 8, 2, 1, 1), (65, 9, 3, 3, 2), (33, 60, 4, 4, 1), (20, 256, 256, 1, 1), (5, 64, 64, 2, 2),
          (40, 130, 12, 2, 1), (70, 64, 1, 32, 1), (12, 256, 100, 4, 2), (200, 192, 10, 64, 5), (4100, 16, 2, 4, 3)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_shapes(shape, score):
    T, E, k, groups, top = shape
    for i, (with_bias, gs, renorm) in enumerate(((False, "max", True), (True, "top2", False), (True, "max", True),
                                                 (False, "top2", False))):
        if gs == "top2" and groups > 1 and E // groups < 2:
            gs = "max"
        _check(_logits(T, E, (F32, BF16, F16, F32)[i], seed=i), k, score, _bias(E) if with_bias else None, groups, top, gs,
               renorm, (1.0, 2.5, -0.5, 16.0)[i])


@pytest.mark.parametrize("T,E,k", [(8193, 64, 6), (8257, 256, 64), (10241, 7, 3), (20001, 256, 8), (65536, 128, 2)])
def test_batches_of_many_segments(T, E, k):
    """More than 128 segments, whose counts come in halves.  The choice without
    groups, of all tokens at once (the scores here are no nearer to each other
    than 64 bits tell)."""
    from bit_quantized_moe_token_amd import moeq
    l, b = _logits(T, E, seed=T), _bias(E)
    for bias in (None, b):
        r = moeq.route_scored(l.cuda(), k, score="sigmoid", bias=None if bias is None else bias.cuda(), scale=2.5)
        s = scores.scores(_np(l).reshape(-1), "sigmoid").reshape(T, E)
        c = _np(l) if bias is None else s + _np(bias)
        ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        off, order, pos = scores.sort_pairs(ids, E)
        assert np.array_equal(r.offsets.cpu().numpy(), off)
        assert np.array_equal(r.sorted_pairs.cpu().numpy(), order) and np.array_equal(r.pair_pos.cpu().numpy(), pos)
        g = np.take_along_axis(s, ids, 1)
        g = 2.5 * g / g.sum(1, keepdims=True)
        assert (np.abs(_np(r.gates) - g) <= 1.01 * 2.0 ** -24 * g).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_strides_and_alignment(dtype):
    _check(_logits(37, 61, dtype), 5, "sigmoid", _bias(61), 1, 1, "max", True, 1.0, strided=True)
    _check(_logits(7, 256, dtype), 5, "softmax", None, 4, 2, "top2", False, 1.0, strided=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [9, 40])
def test_ties_and_near_ties(score, tokens):
    """Equal choices (equal logits and biases) go to the lowest id, choices
    that differ in the last bits of fp32 or below go by their exact order."""
    E = 96
    l = torch.zeros(tokens, E)
    _check(l, 7, score, None, 8, 3, "top2", True, 1.0)
    _check(l, 7, score, torch.zeros(E), 8, 3, "max", True, 1.0)
    l = _logits(tokens, 8).repeat(1, 12)                       # every logit twelve times
    _check(l, 20, score, None, 1, 1, "max", False, 1.0)
    _check(l, 20, score, _bias(8).repeat(12), 4, 2, "top2", True, 1.0)
    # neighbours in fp32 around a score where it is flat: their scores agree in fp32
    step = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t)) for t in range(tokens)])
    l = 9 + step * 2.0 ** -19
    _check(l, 9, score, torch.full((E,), 3.0), 4, 2, "max", True, 1.0)
    _check(l, 9, score, None, 4, 2, "max", True, 1.0)
    # (two sums of such scores can differ by their curvature alone: 2^-42 here, far above 64 bits' rounding)
    _check(3 + step * 2.0 ** -19, 9, score, torch.zeros(E), 4, 2, "top2", True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_of_large_choices_of_opposite_sign(score):
    """Each of a group's two choices is large and their sum is not: what fp32
    loses of them is more than the sums differ by."""
    T, groups = 64, 16
    step = torch.stack([torch.randperm(groups, generator=torch.Generator().manual_seed(t)) for t in range(T)])
    l = torch.zeros(T, groups, 2)
    l[:, :, 0] = step * 2.0 ** (-15 if score == "sigmoid" else -11)     # sums 8e-6 apart, choices of 100 to 7.6e-6
    size = 100.0 + torch.arange(groups) / 7
    bias = torch.stack([size, -size], 1).flatten()
    _check(l.view(T, -1), 4, score, bias, groups, 3, "top2", True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [6, 30])
def test_masked_and_infinite_logits(score, tokens):
    """Experts out of the choice (-infinity, NaN), rows with nothing left,
    the type's lowest value, +infinity."""
    E = 40
    l = _logits(tokens, E)
    l[0] = -INF
    l[1, 3:] = -INF
    l[2, ::2] = -INF
    l[3, 5] = float("nan")
    l[4, 1:] = torch.finfo(F32).min
    l[5] = torch.finfo(F32).min
    bias = _bias(E)
    for b in (None, bias):
        for groups, top, gs in ((1, 1, "max"), (5, 2, "max"), (5, 2, "top2")):
            for renorm in (True, False):
                _check(l, 6, score, b, groups, top, gs, renorm, 1.5)
    _check(torch.full((tokens, E), -INF), 6, score, None, 5, 2, "top2", True, 1.0)
    l = _logits(tokens, E)
    l[0, 7] = l[0, 9] = INF
    l[1] = INF
    l[2, 4] = INF
    _check(l, 6, score, None, 1, 1, "max", True, 1.0)
    _check(l, 6, score, None, 1, 1, "max", False, 1.0)
    b = bias.clone()
    b[3], b[4], b[5] = INF, -INF, float("nan")
    _check(_logits(tokens, E), 6, score, b, 5, 3, "max", True, 1.0)


def test_large_logits_keep_their_ratio():
    """Renormalised gates of logits far from zero: the softmax over the chosen
    needs no score that could underflow; a sigmoid's are formed in 64 bits."""
    l = torch.tensor([[-600.0, -601.0, -602.0, -604.0]]).repeat(20, 1)
    r = _check(l, 2, "sigmoid", None, 1, 1, "max", True, 1.0)
    assert abs(float(r.gates[0, 0]) - 1 / (1 + np.exp(-1.0))) < 1e-6
    l = torch.tensor([[1e4, 1.0, -9e3, -9001.0]]).repeat(20, 1)
    _check(l, 2, "softmax", torch.tensor([-9.0, -9.0, 0.0, 0.0]), 1, 1, "max", True, 1.0)
    _check(-l, 3, "softmax", None, 2, 2, "max", False, 1.0)


def test_no_tokens_and_reused_output():
    from bit_quantized_moe_token_amd import moeq
    r = _check(torch.zeros(0, 12), 3, "softmax", None, 1, 1, "max", True, 1.0)
    assert (r.offsets == 0).all()
    out = moeq.RoutingOut(50, 24, 4, torch.device("cuda", 0))
    for seed in (1, 2):
        before = out.ids._version
        assert _check(_logits(50, 24, seed=seed), 4, "sigmoid", _bias(24), 2, 2, "max", True, 1.0, out=out) is out
        assert out.ids._version > before
    with pytest.raises(ValueError):
        moeq.route_scored(_logits(49, 24).cuda(), 4, out=out)


def test_saved_ids_and_written_offsets():
    """A backward pass that saved a routing's ids and gates is not in the way
    of a caller who uses the other outputs as scratch."""
    from bit_quantized_moe_token_amd import moeq

    class Gates(torch.autograd.Function):
        @staticmethod
        def forward(ctx, l, r):
            ctx.save_for_backward(l, r.ids, r.gates)
            return r.gates.clone()

        @staticmethod
        def backward(ctx, d):
            l, ids, _ = ctx.saved_tensors
            return moeq.route_scored_grad(l, ids, d.contiguous()), None

    l = _logits(30, 16).cuda().requires_grad_()
    for routing in (moeq.route_scored(l.detach(), 3), moeq.route(l.detach(), 3)):
        loss = (Gates.apply(l, routing) ** 2).sum()
        routing.offsets.zero_()
        routing.sorted_pairs.add_(1)
        routing.pair_pos.zero_()
        loss.backward()
        want = moeq.route_scored_grad(l.detach(), routing.ids, 2 * routing.gates)
        assert torch.equal(l.grad, want)
        l.grad = None
        loss = (Gates.apply(l, routing) ** 2).sum()
        routing.ids.zero_()
        with pytest.raises(RuntimeError):          # (what was saved itself)
            loss.backward()


def test_softmax_over_the_chosen_is_the_plain_routing():
    """With renormalised softmax gates the choice is route's, bit for bit in
    the integers, within fp32 in the gates (there 2^-21: fast exponentials)."""
    from bit_quantized_moe_token_amd import moeq
    for T in (9, 500, 5000):
        l = _logits(T, 64).cuda()
        a, b = moeq.route(l, 6), moeq.route_scored(l, 6)
        for n in ("ids", "offsets", "sorted_pairs", "pair_pos"):
            assert torch.equal(getattr(a, n), getattr(b, n))
        assert float((a.gates - b.gates).abs().max()) < 2e-6


def test_refusals():
    from bit_quantized_moe_token_amd import moeq
    l = _logits(4, 16).cuda()
    for kw, e in ((dict(score="relu"), ValueError), (dict(group_score="mean"), ValueError),
                  (dict(bias=torch.zeros(15).cuda()), ValueError),
                  (dict(bias=torch.zeros(16)), TypeError), (dict(bias=torch.zeros(16).half().cuda()), TypeError),
                  (dict(groups=3), moeq.MoeqError), (dict(groups=4, top_groups=5), moeq.MoeqError),
                  (dict(scale=float("nan")), moeq.MoeqError)):
        with pytest.raises(e):
            moeq.route_scored(l, 3, **kw)
    for bad, e in ((l.cpu(), TypeError), (l.double(), TypeError), (l[0], ValueError), (l.T, ValueError)):
        with pytest.raises(e):
            moeq.route_scored(bad, 3)
    with pytest.raises(moeq.MoeqError):
        moeq.route_scored(l, 17)
    ids, dg = torch.zeros(4, 3, dtype=torch.int32).cuda(), torch.zeros(4, 3).cuda()
    for a in ((l.cpu(), ids, dg), (l, ids.long(), dg), (l, ids, dg.half()), (l, ids[:3], dg), (l, ids, dg[:, :2])):
        with pytest.raises((TypeError, ValueError)):
            moeq.route_scored_grad(*a)
    with pytest.raises(TypeError):
        moeq.route_scored_grad(l, ids, dg, out=torch.empty(4, 16).half().cuda())


# ---- gradient

def _check_grad(l, ids, dg, score, renorm, scale, out=None, strided=False):
    """Each entry is a product of factors formed in 64 bits and rounded once
    (half a step); a softmax over all E in fp32: its score (16 * 2^-24 as
    above) times a difference of rounded values (2 more, of its terms)."""
    from bit_quantized_moe_token_amd import moeq
    dev = l.cuda()
    if strided:
        wide = torch.zeros((l.shape[0], l.shape[1] + 5), dtype=l.dtype, device="cuda")
        wide[:, 3:-2] = dev
        dev = wide[:, 3:-2]
    got = moeq.route_scored_grad(dev, ids.int().cuda(), dg.cuda(), score=score, renorm=renorm, scale=scale,
                                 out=dev if out == "in place" else None)
    ref, mag = scores.route_grad(_np(l), ids.numpy(), _np(dg), score, renorm, scale)
    n = 20 if score == "softmax" and not renorm else 2
    tiny = {F32: 2.0 ** -126, F16: 2.0 ** -25, BF16: 2.0 ** -126}[l.dtype]
    bad = np.abs(_np(got) - ref) > torch.finfo(l.dtype).eps / 2 * 1.01 * np.abs(ref) + n * 2.0 ** -24 * mag + tiny
    assert not bad.any(), (int(bad.sum()), float(np.abs(_np(got) - ref).max()))
    return got


def _ids(T, E, k, seed=3):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])


def _dg(T, k, seed=4):
    return torch.randn((T, k), generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_gradient(score, renorm, dtype):
    for T, E, k in ((1, 1, 1), (1, 64, 6), (5, 7, 7), (33, 60, 4), (70, 256, 8), (3, 256, 256), (130, 100, 70), (9, 8, 2),
                    (64, 32, 1), (11, 129, 3)):
        _check_grad(_logits(T, E, dtype), _ids(T, E, k), _dg(T, k), score, renorm, 2.5)
    _check_grad(_logits(21, 61, dtype), _ids(21, 61, 5), _dg(21, 5), score, renorm, -1.0, strided=True)
    _check_grad(_logits(21, 61, dtype), _ids(21, 61, 5), _dg(21, 5), score, renorm, 1.0, out="in place")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_masked_and_extreme_rows(score, renorm):
    T, E, k = 12, 24, 5
    l = _logits(T, E)
    l[0] = -INF
    l[1, 3:] = -INF
    l[2, 5] = float("nan")
    l[3, 1:] = torch.finfo(F32).min
    l[4] = torch.finfo(F32).min
    l[5] *= 30
    l[6, 2] = INF
    ids = _ids(T, E, k)
    ids[7] = torch.tensor([3, 3, 4, 3, 4])            # the same expert twice
    ids[8] = torch.tensor([-1, 24, 2 ** 30, 1, 2])    # no experts
    ids[9] = -7
    got = _check_grad(l, ids, _dg(T, k), score, renorm, 1.0)
    assert (got[0] == 0).all() and (got[9] == 0).all()
    _check_grad(_logits(4, E), _ids(4, E, k), torch.zeros(4, k), score, renorm, 1.0)
    from bit_quantized_moe_token_amd import moeq
    assert moeq.route_scored_grad(torch.zeros(0, 8).cuda(), torch.zeros(0, 2, dtype=torch.int32).cuda(),
                                  torch.zeros(0, 2).cuda()).shape == (0, 8)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_gradient_of_confident_rows(dtype, score, renorm):
    """One expert leads by far, chosen or not, or all gates' gradients are
    equal: every entry is small beside its terms, and is right beside itself.
    Weighted differences in 64 bits; the exponentials of experts outside the
    choice are fp32: 2 steps (2^-22) and the rounding of an argument of up to
    `span` (span * 2^-24), in sums of at most 4 + 6 additions, a quotient and
    two products (20 * 2^-24 in all)."""
    from bit_quantized_moe_token_amd import moeq
    tiny = {F32: 2.0 ** -126, BF16: 2.0 ** -126}[dtype]
    for E, k in ((64, 1), (64, 6), (9, 9), (256, 8), (100, 64), (100, 70), (256, 256)):
        leads = torch.tensor([0.0, 8.0, 12.0, 16.0, 20.0, 30.0, 60.0] * 2)
        T = len(leads)
        l = torch.randn((T, E), generator=torch.Generator().manual_seed(E + k))
        l[:, 3] = leads + l.amax(1)
        l = l.to(dtype)
        ids = _ids(T, E, k)
        for t in range(T):
            if t < T - 2 and 3 not in ids[t]:
                ids[t, k // 2] = 3                     # (the last two as they come)
        for dg in (_dg(T, k), torch.ones(T, k)):
            got = _np(moeq.route_scored_grad(l.cuda(), ids.int().cuda(), dg.cuda(), score=score, renorm=renorm, scale=2.5))
            ref, mag = scores.route_grad_apart(_np(l), ids.numpy(), _np(dg), score, renorm, 2.5)
            span = (_np(l).max(1) - _np(l).min(1))[:, None]
            tol = torch.finfo(dtype).eps / 2 * 1.01 * np.abs(ref) + (20 + span) * 2.0 ** -24 * mag + tiny
            bad = np.abs(got - ref) > tol
            assert not bad.any(), (E, k, int(bad.sum()), float((np.abs(got - ref) / tol).max()))
            if score == "softmax":                     # a row's entries add up to nothing
                assert (np.abs(got.sum(1)) <= tol.sum(1)).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_repeated_experts_in_many_slots(score, renorm):
    """More than 64 slots, some of one expert, some of none; the best expert
    among the repeated ones."""
    T, E, k = 9, 130, 100
    l, ids = _logits(T, E), _ids(T, E, k)
    ids[1, 50:] = ids[1, :50]
    ids[2, ::3] = int(ids[2, 0])
    ids[3, 10], ids[3, 70], ids[3, 99] = -1, 130, 2 ** 30
    ids[4, :] = 7
    for t in (1, 2, 4):
        l[t, ids[t, 0]] = l[t].max() + 2
    _check_grad(l, ids, _dg(T, k), score, renorm, 1.5)
    _check_grad(l, ids, torch.ones(T, k), score, renorm, 1.5)


def test_gradient_against_differences():
    """Of the gates that the forward call returns: central differences with
    steps of 2^-6, whose third-derivative term is below 2^-12 * 2 here, over
    gates rounded to fp32 (2^-24 / 2^-6 each)."""
    from bit_quantized_moe_token_amd import moeq
    T, E, k, h = 20, 12, 3, 2.0 ** -6
    l, dg = _logits(T, E).cuda(), _dg(T, k).cuda()
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        rt = moeq.route_scored(l, k, score=score, renorm=renorm)
        d = moeq.route_scored_grad(l, rt.ids, dg, score=score, renorm=renorm)

        def f(m):
            # the same experts, whatever their order: k = E picks all, the gates are looked up
            r = moeq.route_scored(m, E, score=score, renorm=False)
            s = torch.zeros(T, E, device="cuda").scatter_(1, r.ids.long(), r.gates).gather(1, rt.ids.long()).double()
            return ((s / s.sum(1, keepdim=True) if renorm else s) * dg.double()).sum(1)

        for e in range(E):
            step = torch.zeros(E, device="cuda")
            step[e] = h
            num = (f(l + step) - f(l - step)) / (2 * h)
            assert float((num - d[:, e].double()).abs().max()) < 2.0 ** -10


# ---- streams and graphs

def test_two_streams_and_a_captured_call():
    from bit_quantized_moe_token_amd import moeq
    ls = [_logits(T, 256, seed=T).cuda() for T in (7, 900, 5000)]
    kw = dict(score="sigmoid", bias=_bias(256).cuda(), groups=8, top_groups=4, group_score="top2", scale=2.5)
    names = ("ids", "gates", "offsets", "sorted_pairs", "pair_pos")

    def passes(l):
        r = moeq.route_scored(l, 8, **kw)
        return [getattr(r, n) for n in names] + [moeq.route_scored_grad(l, r.ids, r.gates, score="sigmoid", scale=2.5)]

    ref = [[t.clone() for t in passes(l)] for l in ls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ls]
    got = []
    for _ in range(3):
        for l, st in zip(ls, streams):
            with torch.cuda.stream(st):
                got.append(passes(l))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, ref[i % 3]))
    for l, want in zip(ls, ref):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = passes(l)
        for _ in range(3):
            for t in outs:
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            assert all(torch.equal(a, b) for a, b in zip(passes(l), want))
