"""Scored routing, the experts' products, the combine and the adapters
together, as a model runs them: a block's training step with the router in
it, the low-bit layer under scored routing, and the requests' adapters beside
the 16- and 8-bit projections that they share."""

import numpy as np
import pytest

from oracle import forward, requests, scores
from synth import configs, gen
from tests import layers

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32 = torch.float32


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Block:
    """Router and experts in 16 bits with a shared expert's output beside
    them: x -> y."""

    def __init__(self, dtype=torch.float16, T=70, H=192, I=136, E=16, k=3, seed=0, **kw):
        rng = np.random.default_rng(seed)
        m = lambda *s, scale=1.0: torch.from_numpy(scale * rng.standard_normal(s)).to(dtype).cuda()
        self.T, self.H, self.E, self.k, self.dtype = T, H, E, k, dtype
        self.x, self.shared = m(T, H), m(T, H)
        self.wr = m(1, E, H, scale=H ** -0.5)
        self.w1, self.w2 = m(E, I, H, scale=H ** -0.5), m(E, H, I, scale=I ** -0.5)
        self.kw = dict(score="sigmoid", renorm=True, scale=2.5)
        self.choice = dict(bias=torch.from_numpy(0.01 * rng.standard_normal(E)).float().cuda(), groups=4, top_groups=2,
                           group_score="top2")

    def forward(self):
        from bit_quantized_moe_token_amd import moeq
        logits = moeq.grouped_gemm(self.x, self.wr, None, out_dtype=F32)
        rt = moeq.route_scored(logits, self.k, **self.kw, **self.choice)
        a = moeq.grouped_gemm(self.x, self.w1, rt.offsets, pairs=rt.sorted_pairs, k=self.k)
        z = moeq.grouped_gemm(a, self.w2, rt.offsets)
        y = moeq.combine(z, rt.pair_pos, gates=rt.gates, base=self.shared)
        return dict(logits=logits, rt=rt, a=a, z=z, y=y)

    def backward(self, s, dy):
        from bit_quantized_moe_token_amd import moeq
        rt, k = s["rt"], self.k
        dz, d_gates = moeq.combine_grad(dy, rt.pair_pos, gates=rt.gates, rows=s["z"])
        da = moeq.grouped_gemm(dz, self.w2, rt.offsets, trans=True)
        dxr = moeq.grouped_gemm(da, self.w1, rt.offsets, trans=True)
        dl = moeq.route_scored_grad(s["logits"], rt.ids, d_gates, **self.kw)
        dl16 = dl.to(self.dtype)
        dx = moeq.grouped_gemm(dl16, self.wr, None, trans=True)
        return dict(wr=moeq.grouped_wgrad(dl16, self.x, None),
                    w1=moeq.grouped_wgrad(da, self.x, rt.offsets, pairs=rt.sorted_pairs, k=k),
                    w2=moeq.grouped_wgrad(dz, s["a"], rt.offsets), logits=dl, gates=d_gates,
                    x=moeq.combine(dxr, rt.pair_pos, k=k, base=dx))


def test_training_step_against_autograd():
    """All gradients against double-precision autograd of the same block with
    the same experts.  Stored values are fp16 (half a step 2^-11), fewer than
    ten roundings lie between a gradient and the loss: 10 * 2^-11 of the
    gradient's norm, as in the block without a router."""
    b = Block()
    dy = torch.from_numpy(np.random.default_rng(5).standard_normal((b.T, b.H))).half().cuda()
    s = b.forward()
    got = b.backward(s, dy)
    rt = s["rt"]
    ids, _ = scores.route(_np(s["logits"]), b.k, "sigmoid", _np(b.choice["bias"]), 4, 2, "top2", True, 2.5)
    assert np.array_equal(rt.ids.cpu().numpy(), ids)
    leaf = {n: getattr(b, n).double().cpu().requires_grad_() for n in ("x", "wr", "w1", "w2")}
    logits = leaf["x"] @ leaf["wr"][0].T
    logits.retain_grad()
    sel = torch.sigmoid(logits).gather(1, rt.ids.long().cpu())
    gates = 2.5 * sel / sel.sum(1, keepdim=True)
    gates.retain_grad()
    y = b.shared.double().cpu()
    for j in range(b.k):
        e = rt.ids[:, j].long().cpu()
        a = (leaf["w1"][e] @ leaf["x"][:, :, None])
        y = y + gates[:, j:j + 1] * (leaf["w2"][e] @ a)[:, :, 0]
    assert float((_t(s["y"]) - y.detach()).norm() / y.detach().norm()) < 10 * 2.0 ** -11
    (y * dy.double().cpu()).sum().backward()
    ref = dict({n: v.grad for n, v in leaf.items()}, logits=logits.grad, gates=gates.grad)
    for n, v in ref.items():
        err = float((_t(got[n]).reshape(v.shape) - v).norm() / v.norm())
        assert err < 10 * 2.0 ** -11, (n, err)


def _t(t):
    return t.detach().double().cpu()


@pytest.mark.parametrize("T", [5, 90])
def test_captured_training_step(T):
    """The step in one graph, replayed with eager steps between, gives the
    eager results bit for bit."""
    b = Block(torch.bfloat16, T=T, seed=3)
    dy = torch.randn(b.T, b.H, device="cuda").bfloat16()

    def step():
        s = b.forward()
        g = b.backward(s, dy)
        return [s["y"], s["rt"].ids, s["rt"].gates] + [g[n] for n in sorted(g)]

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
        assert all(torch.equal(a, e) for a, e in zip(outs, eager))
        assert all(torch.equal(a, e) for a, e in zip(step(), eager))


def test_in_an_autograd_function():
    """The calls as one autograd.Function of a caller's: its gradients are
    the calls' own."""
    from bit_quantized_moe_token_amd import moeq
    b = Block(seed=7)

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, z):
            rt = moeq.route_scored(logits, b.k, **b.kw)
            rows = z[rt.sorted_pairs.long() // b.k].contiguous()
            ctx.save_for_backward(logits, rows)
            ctx.rt = rt
            return moeq.combine(rows, rt.pair_pos, gates=rt.gates)

        @staticmethod
        def backward(ctx, dy):
            logits, rows = ctx.saved_tensors
            d_rows, dg = moeq.combine_grad(dy.contiguous(), ctx.rt.pair_pos, gates=ctx.rt.gates, rows=rows)
            return (moeq.route_scored_grad(logits, ctx.rt.ids, dg, **b.kw),
                    moeq.combine(d_rows, ctx.rt.pair_pos, k=b.k))

    logits = torch.randn(b.T, b.E, device="cuda", requires_grad=True)
    z = torch.randn(b.T, b.H, device="cuda", requires_grad=True)
    y = Experts.apply(logits, z)
    # every expert returns the token itself: y = 2.5 x, and the gates' sum has no gradient
    assert torch.allclose(y, 2.5 * z, rtol=1e-6, atol=1e-6)
    y.sum().backward()
    assert torch.allclose(z.grad, torch.full_like(z, 2.5), rtol=1e-6)
    assert float(logits.grad.abs().max()) < 1e-4


@pytest.mark.parametrize("tokens", [3, 64])
def test_low_bit_layer_under_scored_routing(tokens):
    from bit_quantized_moe_token_amd import moeq
    cfg = configs.get("tiny")
    orc = layers.oracle_layer(cfg, 0, cache_blocks=3 * cfg["E"])
    dev = layers.device_layer(cfg, 0, orc)
    x, logits = gen.gen_x(cfg, 0)[:tokens].copy(), gen.gen_logits(cfg, 0)[:tokens].copy()
    kw = dict(score="sigmoid", groups=4, top_groups=2, group_score="max", scale=1.5)
    rt = moeq.route_scored(torch.from_numpy(logits).cuda(), cfg["k"], **kw)
    y = moeq.expert_ffn(dev, torch.from_numpy(x).cuda(), rt, cfg["n_comp"])
    ids, gates = scores.route(logits, cfg["k"], **kw)
    off, order, pos = scores.sort_pairs(ids, cfg["E"])
    ref = forward.moe_forward(orc, x, logits, cfg["k"], cfg["n_comp"],
                              routing=dict(ids=ids, gates=gates, offsets=off, sorted_pairs=order, pair_pos=pos))
    layers.check_y(_np(y), ref, "scored routing")


@pytest.mark.parametrize("tokens", [1, 70])
def test_adapters_beside_the_shared_projections(tokens):
    """The adapters on what linear_i8 and grouped_gemm return, and beside the
    low-bit layer's output, held to the adapters' own rounding."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(9)
    half = lambda *s, scale=1.0: torch.from_numpy(scale * rng.standard_normal(s)).half().cuda()
    K, N, n, R = 256, 320, 4, 16
    x, w = half(tokens, K), half(N, K, scale=K ** -0.5)
    a, b = half(n, R, K, scale=K ** -0.5), half(n, N, R, scale=0.2)
    ids = torch.from_numpy(rng.integers(-1, n, tokens)).int().cuda()
    wq, sw = moeq.quantize_i8(w)
    for y in (moeq.linear_i8(x, wq, sw), moeq.linear_i8(x, wq, sw, out_dtype=F32), moeq.grouped_gemm(x, w[None], None)):
        base = _np(y)
        got = moeq.adapters(x, a, b, ids, y, out=y)
        ref, worst, mag = requests.adapters(_np(x), _np(a), _np(b), ids.tolist(), base)
        kept = 2.0 ** -22 if y.dtype == F32 else 2.0 ** -16
        tol = (1.01 * torch.finfo(y.dtype).eps / 2 * np.abs(ref) + kept * worst
               + (K + R + 4) * 2.0 ** -24 * (mag + np.abs(base)) + 2.0 ** -25)
        assert got is y and (np.abs(_np(got) - ref) <= tol).all()
