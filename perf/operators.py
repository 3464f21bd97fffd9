"""The operators around the low-bit expert layer, as they are measured: products of expert-sorted rows with 16-bit
expert matrices and their two gradients, products in 8-bit integers with one scale per token and per output channel,
and the norms before and after a block with the block's gate and the residual scale, forwards and backwards.

`run` is one pass of one of them: in elementary torch operations while `own` is false, through the framework's public
calls where it is true.  A case's `op` is

  fwd     y[r] = x[pairs[r] // k] W_e^T            for the rows r of every expert e (W_e [n, h])
  dgrad   dx[r] = dy[r] W_e                         (W_e [h, n]: the same rows back through the expert's matrix)
  wgrad   dW_e = sum over e's rows of dy[r]^T x[pairs[r] // k]
  i8      y[r] = sx[t] sw[e] (xq[t] . wq[e]^T),  xq and sx from the token's row x[t], t = pairs[r] // k
          (experts = 0: one matrix and no sorting, t = r)
  norm    r' = alpha r + gate * (w_post * y / rms(y)),  n = w_pre * r' / rms(r'),  rms(v)^2 = mean(v^2) + eps
  norm_grad   the gradients of all inputs of `norm`, from those of r' and n
"""

import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of 16 sequences through the gate (or up) matrices of eight experts kept in 16 bits
        dict(name="experts fwd decode", op="fwd", tokens=16, experts=8, k=2, h=4096, n=14336, skew=1.1, type="f16"),
        # a prefill of 4096 tokens through the same matrices, the busiest expert with ten times the rows of the idlest
        dict(name="experts fwd prefill", op="fwd", tokens=4096, experts=8, k=2, h=4096, n=14336, skew=1.1, type="bf16"),
        # a ragged batch on sizes that are no multiple of a tile
        dict(name="experts fwd odd", op="fwd", tokens=333, experts=16, k=4, h=1000, n=757, skew=0.7, type="f16"),
        # training step of a layer of many small experts: the rows' gradient through the gate matrix
        dict(name="experts dgrad", op="dgrad", tokens=4096, experts=64, k=6, h=1408, n=2048, skew=0.5, type="bf16"),
        # and that of the matrices, in 32 bits for the optimizer
        dict(name="experts wgrad", op="wgrad", tokens=4096, experts=64, k=6, h=2048, n=1408, skew=0.5, type="bf16"),
        # one token through a dense matrix held in 8 bits
        dict(name="int8 one token", op="i8", tokens=1, experts=0, k=1, h=4096, n=14336, skew=0.0, type="f16"),
        # a prefill through the dense down matrix in 8 bits
        dict(name="int8 prefill", op="i8", tokens=4096, experts=0, k=1, h=14336, n=4096, skew=0.0, type="bf16"),
        # 256 tokens on 64 experts in 8 bits: about 24 rows an expert
        dict(name="int8 experts", op="i8", tokens=256, experts=64, k=6, h=2048, n=1408, skew=0.5, type="f16"),
        # odd sizes in 8 bits
        dict(name="int8 odd", op="i8", tokens=201, experts=0, k=1, h=1530, n=1111, skew=0.0, type="bf16"),
        # the two norms between two blocks of one decoded token
        dict(name="norms one token", op="norm", tokens=1, h=4096, type="f16", residual="f16", gate="vector"),
        # and of a long prefill with the residual stream in 32 bits
        dict(name="norms prefill", op="norm", tokens=16384, h=4096, type="bf16", residual="f32", gate="vector"),
        # their gradients in a training step, with a gate of every token's own
        dict(name="norms gradients", op="norm_grad", tokens=8192, h=4096, type="bf16", residual="bf16", gate="token"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A width: spread over the logarithm; half of them multiples of 128 or 16, the others as they come."""
    v, step = _spread(rng, low, high), rng.choice((1, 1, 16, 128))
    return max(low, v // step * step)


def draw(rng):
    op = rng.choice(("fwd", "dgrad", "wgrad", "i8", "i8", "norm", "norm_grad"))
    if op in ("norm", "norm_grad"):
        h = _size(rng, 64, 16384)
        kind = rng.choice(("f16", "bf16"))
        return dict(op=op, tokens=_spread(rng, 1, min(16384, max(1, 2 ** 25 // h))), h=h, type=kind,
                    residual=rng.choice((kind, "f32")), gate=rng.choice(("vector", "token")))
    experts = 0 if op == "i8" and rng.random() < 0.5 else _spread(rng, 2, 128)
    k = rng.randint(1, min(8, experts)) if experts else 1
    h, n = _size(rng, 64, 14336), _size(rng, 64, 14336)
    while max(1, experts) * h * n > 2 ** 28:
        h, n = (max(64, h // 2), n) if h > n else (h, max(64, n // 2))
    rows = min(8192 * k, int(4e11 / (2.0 * h * n)), int(2 ** 27 / max(h, n)))
    return dict(op=op, tokens=_spread(rng, 1, max(1, rows // k)), experts=experts, k=k, h=h, n=n,
                skew=rng.choice((0.0, 0.5, 1.1)) if experts else 0.0, type=rng.choice(("f16", "bf16")))


def _counts(case):
    """Rows of every expert, most first: shares falling with the expert's rank to the power of -skew, whole by the
    largest remainders."""
    rows, e = case["tokens"] * case["k"], case["experts"]
    share = [(i + 1) ** -case["skew"] for i in range(e)]
    want = [rows * s / sum(share) for s in share]
    got = [int(w) for w in want]
    for i in sorted(range(e), key=lambda i: got[i] - want[i])[: rows - sum(got)]:
        got[i] += 1
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind, t, h = TYPES[case["type"]], case["tokens"], case["h"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def activations(rows, width):
        # a hundredth of the channels carries values twenty times the others'
        wide = torch.where(torch.rand(width, generator=g, device=dev) < 0.01, 20.0, 1.0)
        return (normal(rows, width) * wide).to(kind)

    s = dict(case)
    if case["op"] in ("norm", "norm_grad"):
        res = TYPES[case["residual"]]
        s.update(y=activations(t, h), alpha=0.75, w_pre=(1 + 0.2 * normal(h)).to(kind), w_post=(1 + 0.2 * normal(h)).to(kind),
                 gate=(0.5 * normal(*((h,) if case["gate"] == "vector" else (t, h)))).to(kind), res=(3 * normal(t, h)).to(res))
        if case["op"] == "norm_grad":
            s.update(d_res=(0.1 * normal(t, h)).to(res), d_n=(0.1 * normal(t, h)).to(kind))
        return s
    e, k, n = case["experts"], case["k"], case["n"]
    rows = t * k
    if e:
        counts = _counts(case)
        random.Random(seed).shuffle(counts)
        ids = torch.repeat_interleave(torch.arange(e, device=dev), torch.tensor(counts, device=dev))
        order = ids * rows + torch.randperm(rows, generator=g, device=dev)
        s["counts"] = counts
        s["pairs"] = (order.sort().values - ids * rows).int()
        s["offsets"] = torch.tensor([0] + counts, device=dev).cumsum(0).int()
    if case["op"] == "dgrad":
        s["x"] = (0.1 * normal(rows, h)).to(kind)
    else:
        s["x"] = activations(t, h)
    if case["op"] == "wgrad":
        s["dy"] = (0.1 * normal(rows, n)).to(kind)
        return s
    shape = (h, n) if case["op"] == "dgrad" else (n, h)
    w = torch.empty((max(1, e),) + shape, dtype=torch.int8 if case["op"] == "i8" else kind, device=dev)
    if case["op"] == "i8":
        s["ws"] = torch.empty((max(1, e), n), device=dev)
    for i in range(max(1, e)):
        m = normal(*shape) / math.sqrt(h)
        if case["op"] == "i8":
            s["ws"][i] = m.abs().amax(1) / 127
            m = (m / s["ws"][i][:, None]).round()
        w[i] = m
    s["w"] = w
    if case["op"] == "i8" and not e:
        s["w"], s["ws"] = w[0], s["ws"][0]
    return s


# ---- the plain forms

def _rows(s):
    """The source rows of an expert-sorted product, expert by expert."""
    return (s["x"][s["pairs"].long() // s["k"]]).split(s["counts"])


def _plain_fwd(s):
    return torch.cat([x.float() @ w.float().T for x, w in zip(_rows(s), s["w"])]).to(s["x"].dtype)


def _plain_dgrad(s):
    return torch.cat([x.float() @ w.float() for x, w in zip(s["x"].split(s["counts"]), s["w"])]).to(s["x"].dtype)


def _plain_wgrad(s):
    return torch.stack([d.float().T @ x.float() for d, x in zip(s["dy"].split(s["counts"]), _rows(s))])


def _plain_i8(s):
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    q = (x * (127 / top)).round()
    scale = top / 127
    if not s["experts"]:
        return ((q @ s["w"].float().T) * scale * s["ws"]).to(s["x"].dtype)
    at = s["pairs"].long() // s["k"]
    parts = zip(q[at].split(s["counts"]), scale[at].split(s["counts"]), s["w"], s["ws"])
    return torch.cat([(x @ w.float().T) * a * b for x, a, w, b in parts]).to(s["x"].dtype)


def _unit(v):
    inv = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * inv, inv


def _plain_norm(s):
    p = _unit(s["y"].float())[0] * s["w_post"].float()
    r = (s["alpha"] * s["res"].float() + s["gate"].float() * p).to(s["res"].dtype)
    return r, (_unit(r.float())[0] * s["w_pre"].float()).to(s["y"].dtype)


def _plain_norm_grad(s):
    kind, gate, w_post, w_pre = s["y"].dtype, s["gate"].float(), s["w_post"].float(), s["w_pre"].float()
    d_n = s["d_n"].float()
    u, a = _unit(s["res"].float())
    v, b = _unit(s["y"].float())
    c = d_n * w_pre
    dr = s["d_res"].float() + a * (c - u * (c * u).mean(1, keepdim=True))
    c = dr * gate * w_post
    dy = b * (c - v * (c * v).mean(1, keepdim=True))
    d_gate = dr * v * w_post
    return {"d_y": dy.to(kind), "d_residual": (s["alpha"] * dr).to(s["res"].dtype),
            "d_w_pre": (d_n * u).sum(0), "d_w_post": (dr * gate * v).sum(0),
            "d_gate": d_gate.sum(0) if s["gate"].dim() == 1 else d_gate.to(kind)}


PLAIN = {"fwd": _plain_fwd, "dgrad": _plain_dgrad, "wgrad": _plain_wgrad, "i8": _plain_i8, "norm": _plain_norm,
         "norm_grad": _plain_norm_grad}


# ---- the framework's calls

def _own(s):
    from bit_quantized_moe_token_amd import moeq
    op = s["op"]
    if op == "fwd":
        return moeq.grouped_gemm(s["x"], s["w"], s["offsets"], pairs=s["pairs"], k=s["k"])
    if op == "dgrad":
        return moeq.grouped_gemm(s["x"], s["w"], s["offsets"], trans=True)
    if op == "wgrad":
        return moeq.grouped_wgrad(s["dy"], s["x"], s["offsets"], pairs=s["pairs"], k=s["k"], out_dtype=torch.float32)
    if op == "i8":
        if not s["experts"]:
            return moeq.linear_i8(s["x"], s["w"], s["ws"])
        return moeq.linear_i8(s["x"], s["w"], s["ws"], offsets=s["offsets"], pairs=s["pairs"], k=s["k"])
    if op == "norm":
        return moeq.block_norm(s["res"], s["y"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], alpha=s["alpha"],
                               eps=EPS)
    return moeq.block_norm_grad(s["res"], s["d_n"], s["y"], d_res=s["d_res"], w_pre=s["w_pre"], w_post=s["w_post"],
                                gate=s["gate"], alpha=s["alpha"], eps=EPS)


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ---- what a pass cannot do without

def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    t, h, b = case["tokens"], case["h"], size[case["type"]]
    if case["op"] == "norm":
        r = size[case["residual"]]
        gate = t * h * b if case["gate"] == "token" else h * b
        return {"bytes": t * h * (2 * b + 2 * r) + 2 * h * b + gate, "flops": 11.0 * t * h}
    if case["op"] == "norm_grad":
        r = size[case["residual"]]
        gate = 2 * t * h * b if case["gate"] == "token" else h * (b + 4)
        return {"bytes": t * h * (3 * b + 3 * r) + 2 * h * (b + 4) + gate, "flops": 30.0 * t * h}
    n, rows = case["n"], case["tokens"] * case["k"]
    used = sum(c > 0 for c in _counts(case)) if case["experts"] else 1
    flops = 2.0 * rows * h * n
    if case["op"] == "fwd":
        return {"bytes": t * h * b + rows * n * b + used * n * h * b, "flops": flops}
    if case["op"] == "dgrad":
        return {"bytes": rows * (h + n) * b + used * n * h * b, "flops": flops}
    if case["op"] == "wgrad":
        return {"bytes": t * h * b + rows * n * b + case["experts"] * n * h * 4, "flops": flops}
    return {"bytes": t * h * b + rows * n * b + used * n * (h + 4), "flops": flops}


# ---- the same in 64 bits, from the definitions

def _exact_norm(s, d):
    y, r0, gate = d(s["y"]), d(s["res"]), d(s["gate"])
    h = y.shape[1]
    branch = d(s["w_post"]) * y / ((y.square().sum(1) / h + EPS).sqrt())[:, None]
    r = s["alpha"] * r0 + gate * branch
    stored = r.to(s["res"].dtype).double()
    return r, d(s["w_pre"]) * stored / ((stored.square().sum(1) / h + EPS).sqrt())[:, None]


def _through_rms(grad, v):
    """The gradient of v / rms(v) for the incoming grad: grad / rms - v (grad . v) / (h rms^3)."""
    h = v.shape[1]
    rms = (v.square().sum(1, keepdim=True) / h + EPS).sqrt()
    return grad / rms - v * ((grad * v).sum(1, keepdim=True) / (h * rms ** 3)), v / rms


def _exact_norm_grad(s, d):
    y, r, gate, w_post, w_pre, d_n = d(s["y"]), d(s["res"]), d(s["gate"]), d(s["w_post"]), d(s["w_pre"]), d(s["d_n"])
    back, unit_r = _through_rms(d_n * w_pre, r)
    dr = d(s["d_res"]) + back
    dy, unit_y = _through_rms(dr * gate * w_post, y)
    d_gate = dr * w_post * unit_y
    return {"d_y": dy, "d_residual": s["alpha"] * dr, "d_w_pre": (d_n * unit_r).sum(0), "d_w_post": (dr * gate * unit_y).sum(0),
            "d_gate": d_gate.sum(0) if gate.dim() == 1 else d_gate}


def exact(case, seed):
    s = prepare(case, seed)

    def d(v):
        return v.double()

    if case["op"] == "norm":
        return _exact_norm(s, d)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(s, d)
    if case["op"] == "i8" and not case["experts"]:
        step = d(s["x"]).abs().amax(1) / 127
        codes = (d(s["x"]) / step[:, None]).round()
        return (codes * step[:, None]) @ (d(s["w"]) * d(s["ws"])[:, None]).T
    parts, begin = [], 0
    for e, count in enumerate(s["counts"]):
        rows = slice(begin, begin + count)
        begin += count
        source = d(s["x"][rows] if case["op"] == "dgrad" else s["x"][torch.div(s["pairs"][rows].long(), s["k"], rounding_mode="floor")])
        if case["op"] == "wgrad":
            parts.append(d(s["dy"][rows]).T @ source)
        elif case["op"] == "i8":
            step = source.abs().amax(1, keepdim=True) / 127
            parts.append(((source / step).round() * step) @ (d(s["w"][e]) * d(s["ws"][e])[:, None]).T)
        else:
            parts.append(source @ (d(s["w"][e]) if case["op"] == "dgrad" else d(s["w"][e]).T))
    return torch.stack(parts) if case["op"] == "wgrad" else torch.cat(parts)
