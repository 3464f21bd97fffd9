"""The operators of a block together, as a model runs them: the norms around
an expert layer, routing, the experts' products in 16 bits (with the
gradients of a training step), in 8 bits, and the low-bit layer between the
same norms.

References are fp64 on the values that the GPU stored at each step (fp16 or
bf16), so that every stage is held to its own rounding: tolerances are half
steps of the stored type plus fp32 sums, as in the tests of the single
operators, with a factor of 4 for elementwise steps made in torch between
them.
"""

import numpy as np
import pytest

from oracle import norms, products
from synth import configs, gen
from tests import layers

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32 = torch.float32


def _np(t):
    return t.detach().to(F32).cpu().numpy().astype(np.float64)


def _close(got, ref, mag, n, what):
    """|got - ref| within half a step of got's type and n fp32 roundings of
    the magnitudes' sum."""
    eps = torch.finfo(got.dtype).eps / 2
    bad = np.abs(_np(got) - ref) > 1.01 * eps * np.abs(ref) + n * 2.0 ** -23 * mag + 2.0 ** -25
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(_np(got) - ref).max()))


class Experts:
    """A block of experts in 16 bits with its norms: h -> (h', n')."""

    def __init__(self, dtype, T=70, H=192, I=136, E=7, k=2, seed=0):
        from bit_quantized_moe_token_amd import moeq
        rng = np.random.default_rng(seed)
        m = lambda *s, scale=1.0: torch.from_numpy(scale * rng.standard_normal(s)).to(dtype).cuda()
        self.T, self.H, self.I, self.E, self.k, self.dtype = T, H, I, E, k, dtype
        self.h = m(T, H)
        self.w_in = m(H)
        self.wg, self.wu, self.wd = (m(E, n, c, scale=c ** -0.5) for n, c in ((I, H), (I, H), (H, I)))
        self.w_post, self.w_pre, self.gate = m(H), m(H), m(H)
        self.logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
        self.rt = moeq.RoutingOut(T, E, k, self.h.device)

    def forward(self):
        from bit_quantized_moe_token_amd import moeq
        rt, k = self.rt, self.k
        _, n = moeq.block_norm(self.h, w_pre=self.w_in)
        moeq.route(self.logits, k, out=rt)
        kw = dict(pairs=rt.sorted_pairs, k=k)
        g = moeq.grouped_gemm(n, self.wg, rt.offsets, **kw)
        u = moeq.grouped_gemm(n, self.wu, rt.offsets, **kw)
        a = (torch.nn.functional.silu(g.float()) * u.float()).to(self.dtype)
        z = moeq.grouped_gemm(a, self.wd, rt.offsets)                      # [T k, H], sorted
        y = (z.float()[rt.pair_pos.long()].view(self.T, k, self.H) * rt.gates[:, :, None]).sum(1).to(self.dtype)
        h2, n2 = moeq.block_norm(self.h, y, w_pre=self.w_pre, w_post=self.w_post, gate=self.gate, alpha=0.5)
        return dict(n=n, g=g, u=u, a=a, z=z, y=y, h2=h2, n2=n2)

    def backward(self, s, d_h2, d_n2):
        from bit_quantized_moe_token_amd import moeq
        rt, k, T, H = self.rt, self.k, self.T, self.H
        out = moeq.block_norm_grad(s["h2"], d_n2, s["y"], d_res=d_h2, w_pre=self.w_pre, w_post=self.w_post, gate=self.gate,
                                   alpha=0.5)
        pos, tok = rt.sorted_pairs.long(), rt.sorted_pairs.long() // k
        dz = (out["d_y"].float()[tok] * rt.gates.reshape(-1)[pos][:, None]).to(self.dtype)
        da = moeq.grouped_gemm(dz, self.wd, rt.offsets, trans=True, out_dtype=F32)
        g, u = s["g"].float(), s["u"].float()
        sg = torch.sigmoid(g)
        du, dg = (da * g * sg).to(self.dtype), (da * u * sg * (1 + g * (1 - sg))).to(self.dtype)
        kw = dict(pairs=rt.sorted_pairs, k=k)
        out["d_wd"] = moeq.grouped_wgrad(dz, s["a"], rt.offsets)
        out["d_wg"] = moeq.grouped_wgrad(dg, s["n"], rt.offsets, **kw)
        out["d_wu"] = moeq.grouped_wgrad(du, s["n"], rt.offsets, **kw)
        dn = (moeq.grouped_gemm(dg, self.wg, rt.offsets, trans=True, out_dtype=F32) +
              moeq.grouped_gemm(du, self.wu, rt.offsets, trans=True, out_dtype=F32))
        dn = dn[rt.pair_pos.long()].view(T, k, H).sum(1).to(self.dtype)
        first = moeq.block_norm_grad(self.h, dn, w_pre=self.w_in)
        out["d_w_in"] = first["d_w_pre"]
        out["d_h"] = out["d_residual"].float() + first["d_residual"].float()
        return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_forward_stage_by_stage(dtype):
    b = Experts(dtype)
    s = b.forward()
    rt = b.rt
    off, pairs = rt.offsets.cpu().numpy(), rt.sorted_pairs.cpu().numpy()
    P = b.T * b.k
    src = products.source_rows(P, b.T, pairs, b.k)
    _, n = norms.block_norm(_np(b.h), None, _np(b.w_in), None, None, 1.0, 1e-6, True)
    _close(s["n"], n, np.abs(n), b.H, "n")
    for name, w in (("g", b.wg), ("u", b.wu)):
        zero = np.zeros((P, b.I))
        _close(s[name], products.grouped(_np(s["n"]), _np(w), off, src, zero),
               products.grouped(np.abs(_np(s["n"])), np.abs(_np(w)), off, src, zero), b.H, name)
    zero = np.zeros((P, b.H))
    _close(s["z"], products.grouped(_np(s["a"]), _np(b.wd), off, np.arange(P), zero),
           products.grouped(np.abs(_np(s["a"])), np.abs(_np(b.wd)), off, np.arange(P), zero), b.I, "z")
    h2, _ = norms.block_norm(_np(b.h), _np(s["y"]), None, _np(b.w_post), _np(b.gate), 0.5, 1e-6, True)
    _close(s["h2"], h2, np.abs(h2) + np.abs(_np(b.h)), b.H, "h2")
    _, n2 = norms.block_norm(_np(s["h2"]), None, _np(b.w_pre), None, None, 1.0, 1e-6, True)
    _close(s["n2"], n2, np.abs(n2), b.H, "n2")


def test_training_step_against_autograd():
    """All gradients of a step against double-precision autograd of the same
    block.  Stored values are fp16 (half a step 2^-11), about ten roundings lie
    between a gradient and the loss, each of an entry's own size or the size
    of its sum's terms: 10 * 2^-11 of the gradient's norm is the bound."""
    b = Experts(torch.float16, seed=1)
    rng = np.random.default_rng(2)
    d_h2, d_n2 = (torch.from_numpy(rng.standard_normal((b.T, b.H))).half().cuda() for _ in range(2))
    s = b.forward()
    got = b.backward(s, d_h2, d_n2)
    leaf = {n: getattr(b, n).double().cpu().requires_grad_() for n in ("h", "w_in", "wg", "wu", "wd", "w_post", "w_pre", "gate")}
    rms = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    n = rms(leaf["h"]) * leaf["w_in"]
    ids, gates = b.rt.ids.long().cpu(), b.rt.gates.double().cpu()
    y = 0
    for j in range(b.k):
        g = torch.einsum("th,tih->ti", n, leaf["wg"][ids[:, j]])
        u = torch.einsum("th,tih->ti", n, leaf["wu"][ids[:, j]])
        y = y + gates[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(g) * u, leaf["wd"][ids[:, j]])
    h2 = 0.5 * leaf["h"] + leaf["gate"] * leaf["w_post"] * rms(y)
    n2 = rms(h2) * leaf["w_pre"]
    (h2 * d_h2.double().cpu() + n2 * d_n2.double().cpu()).sum().backward()
    names = dict(h="d_h", w_in="d_w_in", wg="d_wg", wu="d_wu", wd="d_wd", w_post="d_w_post", w_pre="d_w_pre", gate="d_gate")
    for k, v in names.items():
        ref = leaf[k].grad.numpy()
        err = np.linalg.norm(_np(got[v]) - ref) / np.linalg.norm(ref)
        assert err < 10 * 2.0 ** -11, (k, err)


def test_captured_training_step():
    """The whole step in one graph, replayed with eager steps between, gives
    the eager results bit for bit."""
    b = Experts(torch.bfloat16, T=33, seed=3)
    d = torch.randn(b.T, b.H, device="cuda").bfloat16()

    def step():
        s = b.forward()
        g = b.backward(s, d, d)
        return [s["h2"], s["n2"]] + [g[k] for k in sorted(g)]

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
        assert all(torch.equal(a, e) for a, e in zip(outs, eager))
        assert all(torch.equal(a, e) for a, e in zip(step(), eager))


@pytest.mark.parametrize("tokens", [1, 64])
def test_low_bit_layer_between_norms_and_int8(tokens):
    """norm -> routing -> low-bit expert layer -> gated norm -> a dense
    matrix in 8 bits, for one decoded token and a batch."""
    from bit_quantized_moe_token_amd import moeq
    cfg = configs.get("tiny")
    orc = layers.oracle_layer(cfg, 0, cache_blocks=3 * cfg["E"])
    dev = layers.device_layer(cfg, 0, orc)
    H, k = cfg["H"], cfg["k"]
    rng = np.random.default_rng(5)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s)).half().cuda()
    h, w_in, w_post, w_pre, gate = half(tokens, H), half(H), half(H), half(H), half(H)
    wq, sw = moeq.quantize_i8(half(300, H))
    logits = gen.gen_logits(cfg, 0)[:tokens].copy()
    _, n = moeq.block_norm(h, w_pre=w_in)
    rt = moeq.route(torch.from_numpy(logits).cuda(), k)
    y = moeq.expert_ffn(dev, n, rt, cfg["n_comp"])
    h2, n2 = moeq.block_norm(h, y, w_pre=w_pre, w_post=w_post, gate=gate, alpha=1.0)
    out = moeq.linear_i8(n2, wq, sw)
    layers.check_y(_np(y), layers.oracle_y(orc, dict(cfg, T=tokens), n.cpu().numpy(), logits, cfg["n_comp"]), "layer")
    ref, _ = norms.block_norm(_np(h), _np(y), None, _np(w_post), _np(gate), 1.0, 1e-6, True)
    _close(h2, ref, np.abs(ref) + np.abs(_np(h)), H, "h2")
    _, ref = norms.block_norm(_np(h2), None, _np(w_pre), None, None, 1.0, 1e-6, True)
    _close(n2, ref, np.abs(ref), H, "n2")
    q, s = products.code_i8(n2.float().cpu().numpy())
    ref = (q.astype(np.float64) @ wq.cpu().numpy().astype(np.float64).T) * s[:, None] * sw.cpu().numpy()
    _close(out, ref, np.abs(ref), 2, "int8")
