"""The operators on both sides of the experts' products, as they are measured: routing by softmax or sigmoid scores with
a bias for balance, groups and renormalised gates, and its gradient; the gate-weighted combine of expert-sorted rows, and
its gradient; and the low-rank adapters of many requests beside a shared projection.

`run` is one pass of one of them: in elementary torch operations while `own` is false, through the framework's public
calls where it is true.  A case's `op` is

  route         s = softmax(l) or sigmoid(l); the k experts with the largest s + bias among those of the best groups;
                gates scale * s_j (/ sum_j s_j), and the pairs (token, slot) sorted by expert
  route_grad    the logits' gradient from the gates'
  combine       out[t] = base[t] + sum_j gates[t, j] rows[pos[t, j]]
  combine_grad  d_rows[pos[t, j]] = gates[t, j] dy[t],  d_gates[t, j] = dy[t] . rows[pos[t, j]]
  adapters      out[r] = y[r] + scale_i B_i (A_i x[r]),  i = ids[r];  out[r] = y[r] where ids[r] = -1
"""

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # a decoding step of 16 sequences over 128 experts, logits as a 16-bit product leaves them
        dict(name="route decode", op="route", tokens=16, experts=128, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renorm=True, scale=1.0, type="bf16"),
        # a prefill over 256 experts in eight groups, balanced by a bias
        dict(name="route prefill", op="route", tokens=8192, experts=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5, type="f32"),
        # training step of a layer of 64 experts, gates not renormalised: every logit has a gradient
        dict(name="route gradient softmax", op="route_grad", tokens=4096, experts=64, k=6, score="softmax", renorm=False,
             scale=1.0, type="f32"),
        # and of 256 experts with renormalised sigmoid gates
        dict(name="route gradient sigmoid", op="route_grad", tokens=16384, experts=256, k=8, score="sigmoid", renorm=True,
             scale=2.5, type="f32"),
        # the experts' rows of a decoding step back to their tokens
        dict(name="combine decode", op="combine", tokens=16, k=2, h=4096, gates=True, base=False, type="f16", out="f16"),
        # those of a prefill, added to the output of a shared expert
        dict(name="combine prefill", op="combine", tokens=4096, k=6, h=2048, gates=True, base=True, type="bf16", out="bf16"),
        # training step: the rows' and the gates' gradients
        dict(name="combine gradients", op="combine_grad", tokens=4096, k=6, h=2048, type="bf16", out="bf16"),
        # a ragged batch, rows of no alignment
        dict(name="combine gradients odd", op="combine_grad", tokens=333, k=4, h=757, type="f16", out="f16"),
        # one decoded token with its request's adapter beside a gate or up matrix
        dict(name="adapters one token", op="adapters", tokens=1, count=64, rank=32, h=4096, n=14336, order="mixed",
             bare=False, ragged=False, type="f16", base="f16"),
        # a decoding step of 64 requests that use 32 adapters of ranks up to 16
        dict(name="adapters decode", op="adapters", tokens=64, count=32, rank=16, h=4096, n=4096, order="mixed", bare=False,
             ragged=True, type="f16", base="f16"),
        # a prefill of eight requests, each with its own adapter
        dict(name="adapters prefill", op="adapters", tokens=4096, count=8, rank=64, h=4096, n=4096, order="runs", bare=False,
             ragged=False, type="bf16", base="bf16"),
        # odd sizes, a projection kept in 32 bits, some requests without an adapter
        dict(name="adapters odd", op="adapters", tokens=333, count=5, rank=13, h=1000, n=757, order="runs", bare=True,
             ragged=False, type="bf16", base="f32"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A width: spread over the logarithm; half of them multiples of 128 or 16, the others as they come."""
    v, step = _spread(rng, low, high), rng.choice((1, 1, 16, 128))
    return max(low, v // step * step)


def draw(rng):
    op = rng.choice(("route", "route", "route_grad", "combine", "combine_grad", "adapters", "adapters"))
    if op in ("route", "route_grad"):
        groups = rng.choice((1, 1, 2, 4, 8)) if op == "route" else 1
        experts = groups * _spread(rng, 2, 256 // groups)
        top_groups = rng.randint(1, groups)
        c = dict(op=op, tokens=_spread(rng, 1, min(65536, 2 ** 21 // experts)), experts=experts,
                 k=rng.randint(1, min(12, top_groups * (experts // groups))), score=rng.choice(("softmax", "sigmoid")),
                 renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)), type=rng.choice(("f32", "f32", "bf16", "f16")))
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_score=rng.choice(("max", "top2")))
        elif c["k"] == 1:      # a single renormalised gate has no gradient
            c["renorm"] = False
        return c
    kind = rng.choice(("f16", "bf16"))
    if op in ("combine", "combine_grad"):
        h, k = _size(rng, 64, 14336), rng.randint(1, 8)
        kind = rng.choice((kind, kind, "f32"))
        c = dict(op=op, tokens=_spread(rng, 1, min(16384, 2 ** 26 // (h * k * SIZE[kind]))), k=k, h=h, type=kind,
                 out=rng.choice((kind, "f32")))
        if op == "combine":
            c.update(gates=rng.random() < 0.7, base=rng.random() < 0.5)
        return c
    count, rank, h, n = _spread(rng, 1, 64), _size(rng, 1, 128), _size(rng, 64, 14336), _size(rng, 64, 14336)
    tokens = _spread(rng, 1, min(4096, 2 ** 25 // (h + 2 * n)))
    return dict(op=op, tokens=tokens, count=count, rank=rank, h=h, n=n, order=rng.choice(("mixed", "runs")),
                bare=rng.random() < 0.3, ragged=rng.random() < 0.5, type=kind, base=rng.choice((kind, kind, "f32")))


def _adapter_rows(case):
    """Adapter of every row before any mixing: rows dealt to the adapters in turn ("mixed") or in runs of falling length;
    with `bare` every eighth row has none."""
    t, n = case["tokens"], case["count"]
    if case["order"] == "mixed":
        ids = [r % n for r in range(t)]
    else:
        share = [(i + 1) ** -0.5 for i in range(n)]
        ids, at = [], 0.0
        for i in range(n):
            at += t * share[i] / sum(share)
            ids += [i] * (min(t, round(at)) - len(ids))
        ids += [n - 1] * (t - len(ids))
    return [-1 if case["bare"] and r % 8 == 7 else i for r, i in enumerate(ids)]


def _ranks(case):
    """Ranks of the adapters: all the same, or falling from it to a quarter."""
    r, n = case["rank"], case["count"]
    return [max(1, r - (3 * r * (i % 4)) // 12) if case["ragged"] else r for i in range(n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind, t = TYPES[case["type"]], case["tokens"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case)
    if case["op"] in ("route", "route_grad"):
        e, k = case["experts"], case["k"]
        # experts differ in how often they are wanted
        s["logits"] = (1.5 * normal(t, e) + normal(e)).to(kind)
        if case["op"] == "route":
            # a bias as balancing leaves it: a whole number of its steps
            s["bias"] = (0.001 * (50 * normal(e)).round()) if case["bias"] else None
        else:
            s["ids"] = s["logits"].float().sort(dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
            s["d_gates"] = normal(t, k)
        return s
    if case["op"] in ("combine", "combine_grad"):
        k, h = case["k"], case["h"]
        s["rows"] = normal(t * k, h).to(kind)
        experts = torch.randint(8 * k, (t * k,), generator=g, device=dev)
        order = experts.sort(stable=True).indices
        s["pos"] = torch.empty(t * k, dtype=torch.int32, device=dev)
        s["pos"][order] = torch.arange(t * k, dtype=torch.int32, device=dev)
        gates = torch.rand((t, k), generator=g, device=dev) + 0.1
        s["gates"] = gates / gates.sum(1, keepdim=True)
        if case["op"] == "combine_grad":
            s["dy"] = (0.1 * normal(t, h)).to(TYPES[case["out"]])
        else:
            if not case["gates"]:
                s["gates"] = None
            s["base"] = normal(t, h).to(TYPES[case["out"]]) if case["base"] else None
        return s
    h, n, count, rank = case["h"], case["n"], case["count"], case["rank"]
    ids = torch.tensor(_adapter_rows(case), device=dev)
    if case["order"] == "mixed":
        ids = ids[torch.randperm(t, generator=g, device=dev)]
    s["ids"] = ids.int()
    wide = torch.where(torch.rand(h, generator=g, device=dev) < 0.01, 20.0, 1.0)
    s["x"] = (normal(t, h) * wide).to(kind)
    s["y"] = (3 * normal(t, n)).to(TYPES[case["base"]])
    s["a"] = (normal(count, rank, h) / math.sqrt(h)).to(kind)
    s["b"] = (0.1 * normal(count, n, rank)).to(kind)
    s["scale"] = 0.5 + torch.rand(count, generator=g, device=dev)
    s["rank_of"] = _ranks(case)
    s["ranks"] = None
    if case["ragged"]:
        s["ranks"] = torch.tensor(s["rank_of"], dtype=torch.int32, device=dev)
        beyond = torch.arange(rank, device=dev) >= s["ranks"][:, None]
        s["a"][beyond] = 0
        s["b"].transpose(1, 2)[beyond] = 0
    # which adapters have rows, and which: the program knows who asked
    s["rows_of"] = [(i, torch.nonzero(ids == i).flatten()) for i in sorted(set(_adapter_rows(case)) - {-1})]
    return s


# ---- the plain forms

def _scores(l, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    u = torch.exp(l - l.amax(1, keepdim=True))
    return u / u.sum(1, keepdim=True)


def _plain_route(s):
    # 64 bits: which expert comes first may hang on the last bits of two scores
    l = s["logits"].double()
    t, e = l.shape
    score = _scores(l, s["score"])
    if s["bias"] is not None:
        choice = group = score + s["bias"].double()
    else:                    # the scores' order is that of the logits
        choice, group = l, score if s["group_score"] == "top2" else l
    if s["groups"] > 1:
        group = group.view(t, s["groups"], -1).sort(dim=2, descending=True).values
        best = group[:, :, 0] if s["group_score"] == "max" else group[:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        inside = torch.zeros_like(best).scatter_(1, kept, 1.0).repeat_interleave(e // s["groups"], 1)
        choice = torch.where(inside > 0, choice, -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    gates = score.gather(1, ids)
    if s["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    flat = ids.flatten()
    order = flat.sort(stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    ends = (flat[:, None] == torch.arange(e, device=flat.device)).sum(0).cumsum(0)
    return {"ids": ids.int(), "gates": (s["scale"] * gates).float(), "offsets": torch.cat([ends.new_zeros(1), ends]).int(),
            "sorted_pairs": order.int(), "pair_pos": pos.int()}


def _plain_route_grad(s):
    l, ids, dg = s["logits"].float(), s["ids"].long(), s["d_gates"]
    score = _scores(l, s["score"])
    chosen = score.gather(1, ids)
    if s["renorm"]:
        total = chosen.sum(1, keepdim=True)
        v = s["scale"] * (dg - (dg * chosen).sum(1, keepdim=True) / total) / total
    else:
        v = s["scale"] * dg
    d = torch.zeros_like(l).scatter_(1, ids, v)
    if s["score"] == "sigmoid":
        d = d * score * (1 / (1 + torch.exp(l)))
    else:
        d = score * (d - (v * chosen).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _plain_combine(s):
    t, k = s["tokens"], s["k"]
    rows = s["rows"][s["pos"].long()].view(t, k, -1).float()
    if s["gates"] is not None:
        rows = rows * s["gates"][:, :, None]
    out = rows.sum(1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(TYPES[s["out"]])


def _plain_combine_grad(s):
    t, k = s["tokens"], s["k"]
    dy, pos = s["dy"].float(), s["pos"].long()
    d_rows = torch.empty_like(s["rows"])
    d_rows[pos] = (dy[:, None, :] * s["gates"][:, :, None]).to(s["rows"].dtype).view(t * k, -1)
    return {"d_rows": d_rows, "d_gates": (s["rows"][pos].float().view(t, k, -1) * dy[:, None, :]).sum(2)}


def _plain_adapters(s):
    out = s["y"].clone()
    for i, rows in s["rows_of"]:
        r = s["rank_of"][i]
        z = s["x"][rows].float() @ s["a"][i, :r].float().T
        d = s["scale"][i] * (z @ s["b"][i, :, :r].float().T)
        out[rows] = (s["y"][rows].float() + d).to(out.dtype)
    return out


PLAIN = {"route": _plain_route, "route_grad": _plain_route_grad, "combine": _plain_combine,
         "combine_grad": _plain_combine_grad, "adapters": _plain_adapters}


# ---- the framework's calls

def _own(s):
    from bit_quantized_moe_token_amd import moeq
    op = s["op"]
    if op == "route":
        r = moeq.route_scored(s["logits"], s["k"], score=s["score"], bias=s["bias"], groups=s["groups"],
                              top_groups=s["top_groups"], group_score=s["group_score"], renorm=s["renorm"], scale=s["scale"])
        return {"ids": r.ids, "gates": r.gates, "offsets": r.offsets, "sorted_pairs": r.sorted_pairs, "pair_pos": r.pair_pos}
    if op == "route_grad":
        return moeq.route_scored_grad(s["logits"], s["ids"], s["d_gates"], score=s["score"], renorm=s["renorm"],
                                      scale=s["scale"])
    if op == "combine":
        return moeq.combine(s["rows"], s["pos"], gates=s["gates"], k=s["k"], base=s["base"], out_dtype=TYPES[s["out"]])
    if op == "combine_grad":
        d_rows, d_gates = moeq.combine_grad(s["dy"], s["pos"], gates=s["gates"], rows=s["rows"])
        return {"d_rows": d_rows, "d_gates": d_gates}
    return moeq.adapters(s["x"], s["a"], s["b"], s["ids"], s["y"], scale=s["scale"], ranks=s["ranks"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ---- what a pass cannot do without

def work(case):
    t = case["tokens"]
    if case["op"] in ("route", "route_grad"):
        e, k, b = case["experts"], case["k"], SIZE[case["type"]]
        if case["op"] == "route":
            return {"bytes": t * e * b + 16 * t * k + 4 * (e + 1) + 4 * e * case["bias"], "flops": 10.0 * t * e}
        return {"bytes": 2 * t * e * b + 8 * t * k, "flops": 10.0 * t * e}
    if case["op"] == "combine":
        k, h, o = case["k"], case["h"], SIZE[case["out"]]
        return {"bytes": t * h * (k * SIZE[case["type"]] + o * (1 + case["base"])) + t * k * (4 + 4 * case["gates"]),
                "flops": 2.0 * t * k * h}
    if case["op"] == "combine_grad":
        k, h = case["k"], case["h"]
        return {"bytes": t * h * (2 * k * SIZE[case["type"]] + SIZE[case["out"]]) + 12 * t * k, "flops": 3.0 * t * k * h}
    h, n = case["h"], case["n"]
    ids, rank = _adapter_rows(case), _ranks(case)
    with_one = [i for i in ids if i >= 0]
    return {"bytes": len(with_one) * h * 2 + 2 * t * n * SIZE[case["base"]] + 4 * t + sum(rank[i] for i in set(with_one)) * (h + n) * 2,
            "flops": sum(2.0 * rank[i] * (h + n) for i in with_one)}


# ---- the same in 64 bits, from the definitions

def _exact_score(l, score):
    if score == "sigmoid":
        return torch.special.expit(l)
    return torch.exp(l - torch.logsumexp(l, 1, keepdim=True))


def _exact_route(s):
    """One expert after the other: the best of those left, the lowest of equal ones."""
    l = s["logits"].double()
    t, e = l.shape
    score, size = _exact_score(l, s["score"]), e // s["groups"]
    left = l.clone() if s["bias"] is None else score + s["bias"].double()
    if s["groups"] > 1:
        ranked = (score if s["bias"] is None and s["group_score"] == "top2" else left).view(t, s["groups"], size)
        worth = torch.topk(ranked, 1 if s["group_score"] == "max" else 2, 2).values.sum(2)
        out = torch.ones_like(worth, dtype=torch.bool)
        for _ in range(s["top_groups"]):
            best = (worth == worth.amax(1, keepdim=True)).float().argmax(1)
            out[torch.arange(t), best], worth[torch.arange(t), best] = False, -math.inf
        left[out.repeat_interleave(size, 1)] = -math.inf
    ids = []
    for _ in range(s["k"]):
        first = (left == left.amax(1, keepdim=True)) * torch.arange(e, 0, -1, device=l.device)
        ids.append(first.argmax(1))
        left[torch.arange(t), ids[-1]] = -math.inf
    gates = torch.stack([score[torch.arange(t), i] for i in ids], 1)
    if s["renorm"]:
        gates /= gates.sum(1, keepdim=True)
    return {"ids": None, "gates": gates * s["scale"], "offsets": None, "sorted_pairs": None, "pair_pos": None}


def _exact_route_grad(s):
    """Through double-precision autograd of the gates."""
    l = s["logits"].double().requires_grad_()
    with torch.enable_grad():
        gates = _exact_score(l, s["score"]).gather(1, s["ids"].long())
        if s["renorm"]:
            gates = gates / gates.sum(1, keepdim=True)
        return torch.autograd.grad((s["scale"] * gates * s["d_gates"].double()).sum(), l)[0]


def exact(case, seed):
    s = prepare(case, seed)
    op, t = case["op"], case["tokens"]
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    if op == "combine":
        out = torch.zeros((t, case["h"]), dtype=torch.float64, device="cuda") if s["base"] is None else s["base"].double()
        for j in range(case["k"]):
            r = s["rows"].double()[s["pos"].view(t, -1)[:, j].long()]
            out += r if s["gates"] is None else r * s["gates"].double()[:, j:j + 1]
        return out
    if op == "combine_grad":
        rows = s["rows"].double().requires_grad_()
        gates = s["gates"].double().requires_grad_()
        with torch.enable_grad():
            y = sum(rows[s["pos"].view(t, -1)[:, j].long()] * gates[:, j:j + 1] for j in range(case["k"]))
            d_rows, d_gates = torch.autograd.grad((y * s["dy"].double()).sum(), (rows, gates))
        return {"d_rows": d_rows, "d_gates": d_gates}
    out = s["y"].double()
    for i in range(case["count"]):
        mine = s["ids"] == i
        m = s["b"][i].double() @ s["a"][i].double()          # [n, h]: the adapter as one matrix
        out[mine] += float(s["scale"][i]) * (s["x"][mine].double() @ m.T)
    return out
