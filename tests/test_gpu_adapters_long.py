"""The adapters in long batches, where the first kernel takes 32 rows a
workgroup (from 2048 rows on) and a workgroup of the second goes over its
outputs in several turns; and the bits of z = A x that are kept.

Bounds as in the tests of short batches, but what z is kept to is what the
header says: 2^-16 of the row's largest z beside bf16 outputs, 2^-22 beside
fp16 ones, 2^-24 beside fp32."""

import numpy as np
import pytest

from oracle import requests

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)]
KEPT = {F32: 2.0 ** -24, F16: 2.0 ** -22, BF16: 2.0 ** -16}
IDS = lambda v: "-".join(str(d).split(".")[-1] for d in v) if isinstance(v, tuple) and isinstance(v[0], torch.dtype) else str(v)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _case(T, n, R, K, N, types, order, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)
    ids = torch.randint(-1, n, (T,), generator=g).int()
    if order == "runs":
        ids = ids.sort().values
    return dict(x=rand(T, K).to(types[0]), a=(rand(n, R, K) * K ** -0.5).to(types[0]), b=(0.2 * rand(n, N, R)).to(types[0]),
                ids=ids, y=(3 * rand(T, N)).to(types[1]), scale=0.5 + torch.rand((n,), generator=g),
                ranks=torch.randint(0, R + 1, (n,), generator=g).int())


def _check(c, got):
    K, R = c["x"].shape[1], c["a"].shape[1]
    scale, ranks = c.get("scale"), c.get("ranks")
    ref, worst, mag = requests.adapters_of_many_rows(_np(c["x"]), _np(c["a"]), _np(c["b"]), c["ids"].numpy(), _np(c["y"]),
                                                     None if scale is None else scale.tolist(),
                                                     None if ranks is None else ranks.tolist())
    tol = (1.01 * torch.finfo(got.dtype).eps / 2 * np.abs(ref) + (K + 1) * 2.0 ** -24 * mag + KEPT[got.dtype] * worst
           + (R + 3) * 2.0 ** -24 * (mag + np.abs(_np(c["y"]))) + (2.0 ** -25 if got.dtype == F16 else 2.0 ** -126))
    bad = ~(np.abs(_np(got) - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(_np(got) - ref) / tol)))
    none = c["ids"] < 0
    assert torch.equal(got.cpu()[none], c["y"][none])


def _call(c, **kw):
    from bit_quantized_moe_token_amd import moeq
    return moeq.adapters(**{k: v.cuda() for k, v in c.items()}, **kw)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("R", [13, 16, 32, 33, 64, 100, 256])
def test_both_sides_of_the_switch(types, R):
    for T, order, K, N, plain in ((2047, "mixed", 100, 48, False), (2048, "runs", 264, 48, True), (2049, "mixed", 5, 40, True),
                                  (2063, "runs", 200, 72, False), (2065, "mixed", 129, 56, False), (2080, "runs", 64, 8, True)):
        c = _case(T, 5, R, K, N, types, order, seed=R)
        if plain:
            del c["scale"], c["ranks"]
        _check(c, _call(c))


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("R", [16, 32, 40, 128, 200])
def test_several_turns_of_outputs(types, R):
    """Outputs beyond what one round of workgroups takes in one turn, with a
    ragged last turn, in tiles that one and several adapters share."""
    for T, order, N in ((2065, "runs", 2611), (1500, "mixed", 3336), (700, "runs", 8219)):
        _check(c := _case(T, 3, R, 72, N, types, order, seed=R), _call(c))


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_strides_and_alignment(types):
    """No alignment beyond an element's, NaN all around; in place."""
    from bit_quantized_moe_token_amd import moeq

    def inside(t, pad, at):
        wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., at:at + t.shape[-1]] = t.cuda()
        return wide[..., at:at + t.shape[-1]]

    for T, R, K, N in ((2065, 11, 125, 2307), (2050, 72, 131, 99)):
        c = _case(T, 3, R, K, N, types, "mixed")
        x, a, b, y = inside(c["x"], 3, 1), inside(c["a"], 1, 1), inside(c["b"], 5, 2), inside(c["y"], 7, 3)
        out = inside(torch.zeros_like(c["y"]), 4, 1)
        rest = dict(scale=c["scale"].cuda(), ranks=c["ranks"].cuda())
        assert moeq.adapters(x, a, b, c["ids"].cuda(), y, out=out, **rest) is out
        _check(c, out)
        whole = torch.as_strided(out, (T, N + 4), (N + 4, 1), out.storage_offset() - 1)
        assert torch.isnan(whole[:, 0]).all() and torch.isnan(whole[:, N + 1:]).all()
        moeq.adapters(x, a, b, c["ids"].cuda(), y, out=y, **rest)
        assert torch.equal(y, out)


def test_infinities_stay_in_their_rows():
    """In both halves of a tile of 32 rows, and what no row uses."""
    c = _case(2100, 4, 20, 72, 64, (BF16, BF16), "mixed")
    c["ranks"] = torch.tensor([5, 20, 9, 3]).int()
    want = _call(c)
    _check(c, want)
    hit = [3, 21, 40, 1056, 2099]
    c["x"][hit, 7] = float("inf")
    c["x"][c["ids"] < 0] = float("nan")
    c["a"][0, 5:], c["b"][0, :, 5:] = float("nan"), float("inf")
    got = _call(c)
    keep = [r for r in range(2100) if r not in hit]
    assert torch.equal(got[keep], want[keep])
    assert not any(torch.isfinite(got[r]).any() for r in hit if c["ids"][r] >= 0)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("T", [1, 37, 2100])
def test_bits_of_z(types, T):
    """Every z is a number of 24 bits that its three products sum to exactly,
    every output is one of them on top of y: what is lost is what z is kept
    to.  Beside 16 bits y takes z away but for what its type cannot hold."""
    g = torch.Generator().manual_seed(T)
    n, R, N = 2, 20, 48
    m = torch.randint(128, 251, (n, R, 3), generator=g)
    a = m / 128 * torch.pow(2.0, -(torch.arange(R) % 5))[None, :, None]          # [1, 2) and below
    x = torch.tensor([2.0 ** 4, 2.0 ** -4, 2.0 ** -12])[None] * torch.pow(2.0, torch.arange(T) % 3)[:, None]
    b = torch.zeros(n, N, R)
    b[:, torch.arange(N), torch.arange(N) % R] = 1.0
    ids = (torch.arange(T) % n).int()
    z = torch.einsum("rk,rjk->rj", x.double(), a.double()[ids.long()])[:, torch.arange(N) % R]
    y = torch.zeros(T, N) if types[1] == F32 else -z.to(types[1])
    c = dict(x=x.to(types[0]), a=a.to(types[0]), b=b.to(types[0]), ids=ids, y=y)
    assert (c["x"].double() == x.double()).all() and (c["a"].double() == a.double()).all() and (z == z.float()).all()
    want = (z + y.double()).numpy()
    off = np.abs(_np(_call(c)) - want)
    top = z.abs().amax(1, keepdim=True).numpy()
    assert (off <= KEPT[types[1]] * top + 1.01 * torch.finfo(types[1]).eps / 2 * np.abs(want)
            + (2.0 ** -25 if types[1] == F16 else 0)).all(), float((off / top).max())


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("T", [40, 2100])
def test_infinities_in_b_stay_in_their_outputs(types, T):
    """Of the adapter that has them, in the column they belong to, and not
    beyond its rank."""
    c = _case(T, 3, 20, 72, 70, types, "mixed")
    c["ranks"] = torch.tensor([20, 12, 20]).int()
    want = _call(c)
    c["b"][1, 33, 4], c["b"][1, 60, 15] = float("inf"), float("-inf")       # (the second beyond the rank)
    got = _call(c)
    hit = torch.zeros(T, 70, dtype=torch.bool)
    hit[c["ids"] == 1, 33] = True
    assert not torch.isfinite(got.cpu()[hit]).any() and hit.any()
    assert torch.equal(got.cpu()[~hit], want.cpu()[~hit])
