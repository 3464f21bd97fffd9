"""The combine of expert-sorted rows and its gradients against the fp64 forms:
outputs within half a step of their type and one fp32 rounding per term of a
sum, of the terms' magnitudes."""

import numpy as np
import pytest

from oracle import products

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
PAIRS = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F16), (F32, BF16), (F32, F32)]
IDS = lambda v: "-".join(str(d).split(".")[-1] for d in v) if isinstance(v, tuple) and isinstance(v[0], torch.dtype) else str(v)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _rand(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _strided(t, pad, at):
    """t on the GPU as part of wider rows (NaN beside it)."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, at:at + t.shape[1]] = t.cuda()
    return wide[:, at:at + t.shape[1]]


def _close(got, ref, mag, n, what):
    dtype = got.dtype
    tiny = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -134}[dtype]
    bad = np.abs(_np(got) - ref) > 1.01 * torch.finfo(dtype).eps / 2 * np.abs(ref) + n * 1.01 * 2.0 ** -24 * mag + tiny
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(_np(got) - ref))))


def _positions(T, k, P, seed=0):
    """Distinct positions of T * k pairs among P rows; with too few rows some pairs have none."""
    g = torch.Generator().manual_seed(seed)
    return torch.cat([torch.randperm(P, generator=g), torch.full((max(0, T * k - P),), -1)])[:T * k].int()


SIZES = [(1, 1, 1), (1, 2, 4096), (3, 8, 7), (5, 1, 64), (17, 2, 100), (4, 6, 2048), (2, 3, 2053), (33, 4, 757), (300, 5, 48),
         (2, 2, 8200), (1, 256, 40), (6, 16, 24)]


@pytest.mark.parametrize("types", PAIRS, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_combine(types, size):
    from bit_quantized_moe_token_amd import moeq
    (tr, to), (T, k, N) = types, size
    P = T * k + 3
    rows, base, pos = _rand((P, N), tr, 1), _rand((T, N), to, 2), _positions(T, k, P)
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(3))
    for g, b in ((gates, base), (gates, None), (None, base), (None, None)):
        got = moeq.combine(rows.cuda(), pos.cuda(), gates=g.cuda() if g is not None else None, k=k,
                           base=b.cuda() if b is not None else None, out_dtype=to)
        ref, mag = products.combine(_np(rows), pos.numpy(), g, None if b is None else _np(b), T, k)
        assert got.dtype == to
        _close(got, ref, mag, k + 1, (g is None, b is None))


@pytest.mark.parametrize("types", PAIRS, ids=IDS)
def test_strides_in_place_and_missing_pairs(types):
    from bit_quantized_moe_token_amd import moeq
    tr, to = types
    T, k, N, P = 19, 3, 203, 40                # 57 pairs, 40 rows
    rows, base, pos = _rand((P, N), tr, 4), _rand((T, N), to, 5), _positions(T, k, P, 6)
    pos[5], pos[7] = P, 2 ** 31 - 1
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(7))
    ref, mag = products.combine(_np(rows), pos.numpy(), gates, _np(base), T, k)
    b = _strided(base, 5, 3)
    out = _strided(torch.zeros(T, N, dtype=to), 9, 1)
    assert moeq.combine(_strided(rows, 6, 1), pos.cuda(), gates=gates.cuda(), base=b, out=out) is out
    _close(out, ref, mag, k + 1, "strided")
    whole = torch.as_strided(out, (T, N + 9), (N + 9, 1), out.storage_offset() - 1)
    assert torch.isnan(whole[:, 0]).all() and torch.isnan(whole[:, N + 1:]).all()      # nothing beside the rows
    before = b._version
    moeq.combine(rows.cuda(), pos.cuda(), gates=gates.cuda(), base=b, out=b)
    assert torch.equal(b, out) and b._version > before
    # rows and gates of pairs left out do not matter
    bad = rows.clone()
    bad[pos[0]] = float("nan")
    some = pos.clone()
    some[0] = -1
    gates[0, 0] = float("inf")
    got = moeq.combine(bad.cuda(), some.cuda(), gates=gates.cuda(), out_dtype=to)
    assert torch.isfinite(got).all()


def test_empty():
    from bit_quantized_moe_token_amd import moeq
    rows, pos = torch.ones(4, 8).half().cuda(), torch.full((6,), -1, dtype=torch.int32).cuda()
    assert moeq.combine(rows, pos[:0], k=2).shape == (0, 8)
    assert (moeq.combine(rows, pos, k=2) == 0).all()                       # no pair anywhere
    assert (moeq.combine(rows[:0], pos, k=2) == 0).all()                   # no rows at all
    d, dg = moeq.combine_grad(torch.ones(3, 8).half().cuda(), pos, gates=torch.ones(3, 2).cuda(), rows=rows,
                              out=torch.full((4, 8), 5.0).half().cuda())
    assert (d == 5).all() and (dg == 0).all()
    d, dg = moeq.combine_grad(torch.ones(0, 8).half().cuda(), pos[:0], gates=torch.ones(0, 2).cuda(), rows=rows)
    assert d.shape == (4, 8) and dg.shape == (0, 2)


@pytest.mark.parametrize("types", PAIRS, ids=IDS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradients(types, size):
    from bit_quantized_moe_token_amd import moeq
    (tr, to), (T, k, N) = types, size
    P = T * k + 2
    rows, dy, pos = _rand((P, N), tr, 1), _rand((T, N), to, 2, 0.1), _positions(T, k, P)
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(3))
    before = torch.full((P, N), 7.0, dtype=tr)
    args = (dy.cuda(), pos.cuda())
    d_rows, d_gates = moeq.combine_grad(*args, gates=gates.cuda(), rows=rows.cuda(), out=before.cuda())
    ref_r, ref_g, mag = products.combine_grad(_np(dy), pos.numpy(), gates, _np(rows), P, _np(before))
    _close(d_rows, ref_r, np.abs(ref_r), 1, "d_rows")
    # products of 16-bit values are exact in fp32, of 32-bit ones fused or rounded; N additions
    _close(d_gates, ref_g, mag, N + 1, "d_gates")
    # without the gates' gradient, and without gates
    only, none = moeq.combine_grad(*args, gates=gates.cuda(), out=before.cuda())
    assert none is None and torch.equal(only, d_rows)
    if pos.max() < T * k:
        assert torch.equal(moeq.combine_grad(*args, gates=gates.cuda(), out_dtype=tr)[0], d_rows[:T * k])
    plain, none = moeq.combine_grad(*args, k=k, rows=rows.cuda())
    ref, _, _ = products.combine_grad(_np(dy), pos.numpy(), torch.ones(T, k), None, P, np.zeros((P, N)))
    assert none is None
    _close(plain.cpu()[pos.long()], ref[pos.numpy()], np.abs(ref[pos.numpy()]), 1, "no gates")


@pytest.mark.parametrize("types", PAIRS, ids=IDS)
def test_gradients_strided_and_missing(types):
    from bit_quantized_moe_token_amd import moeq
    tr, to = types
    T, k, N, P = 19, 3, 203, 40
    rows, dy, pos = _rand((P, N), tr, 4), _rand((T, N), to, 5), _positions(T, k, P, 6)
    pos[5], pos[7], gone = P, 2 ** 31 - 1, pos[[5, 7]].clone()
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(7))
    out = _strided(torch.full((P, N), 3.0, dtype=tr), 9, 1)
    d_rows, d_gates = moeq.combine_grad(_strided(dy, 5, 3), pos.cuda(), gates=gates.cuda(), rows=_strided(rows, 6, 1), out=out)
    ref_r, ref_g, mag = products.combine_grad(_np(dy), pos.numpy(), gates, _np(rows), P, np.full((P, N), 3.0))
    assert d_rows is out and set(gone.tolist()) - set(pos.tolist())
    _close(d_rows, ref_r, np.abs(ref_r), 1, "d_rows")
    _close(d_gates, ref_g, mag, N + 1, "d_gates")
    whole = torch.as_strided(out, (P, N + 9), (N + 9, 1), out.storage_offset() - 1)
    assert torch.isnan(whole[:, 0]).all() and torch.isnan(whole[:, N + 1:]).all()


def test_gradients_against_differences():
    """combine is linear in each input: the difference over a step of one
    value is the gradient up to fp32 sums (k + N terms of a few units)."""
    from bit_quantized_moe_token_amd import moeq
    T, k, N = 3, 2, 10
    rows, dy, pos = _rand((6, N), F32, 1).cuda(), _rand((T, N), F32, 2).cuda(), _positions(T, k, 6).cuda()
    gates = torch.rand((T, k)).cuda()
    d_rows, d_gates = moeq.combine_grad(dy, pos, gates=gates, rows=rows)
    f = lambda r, g: float((moeq.combine(r, pos, gates=g).double() * dy.double()).sum())
    for i in range(6):
        step = torch.zeros_like(rows)
        step[i, 3 + i % 3] = 1.0
        assert abs((f(rows + step, gates) - f(rows - step, gates)) / 2 - float(d_rows[i, 3 + i % 3])) < 1e-5
        step = torch.zeros_like(gates)
        step.view(-1)[i] = 1.0
        assert abs((f(rows, gates + step) - f(rows, gates - step)) / 2 - float(d_gates.view(-1)[i])) < 1e-5


def test_rows_beyond_32_bit_offsets():
    """Rows whose bytes and elements lie beyond 2^32 of the base."""
    from bit_quantized_moe_token_amd import moeq
    N, P = 1 << 20, 4200                              # 8.8 GB
    rows = torch.zeros((P, N), dtype=F16, device="cuda")
    pos = torch.tensor([P - 1, 3, 4097, P - 2], dtype=torch.int32)
    vals = torch.randint(-8, 8, (4, N), generator=torch.Generator().manual_seed(0)).half()
    rows[pos.long().cuda()] = vals.cuda()
    gates = torch.tensor([[0.5, 0.25], [1.0, 2.0]])
    got = moeq.combine(rows, pos.cuda(), gates=gates.cuda())
    want = torch.stack([0.5 * vals[0].float() + 0.25 * vals[1].float(), vals[2].float() + 2 * vals[3].float()]).half()
    assert torch.equal(got.cpu(), want)
    d, dg = moeq.combine_grad(want.cuda(), pos.cuda(), gates=gates.cuda(), rows=rows, out=rows.zero_())
    assert torch.equal(d[P - 1].cpu(), (0.5 * want[0].float()).half()) and torch.equal(d[P - 2].cpu(), (2 * want[1].float()).half())


@pytest.mark.parametrize("types", PAIRS, ids=IDS)
@pytest.mark.parametrize("T", [1075, 1100])
def test_rows_on_both_sides_of_the_caches(types, T):
    """Rows of a little less and a little more than 80 MiB, which are read in
    different ways, with a ragged end and pairs that point nowhere."""
    from bit_quantized_moe_token_amd import moeq
    tr, to = types
    k, N = 8, 2429 if tr == F32 else 4858
    P = T * k - 5
    size = 4 if tr == F32 else 2
    assert (T * k * N * size > 80 << 20) == (T == 1100)
    rows, base, pos = _rand((P, N), tr, 1), _rand((T, N), to, 2), _positions(T, k, P)
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(3))
    got = moeq.combine(rows.cuda(), pos.cuda(), gates=gates.cuda(), base=base.cuda())
    ref, mag = products.combine(_np(rows), pos.numpy(), gates, _np(base), T, k)
    _close(got, ref, mag, k + 1, "out")
    d_rows, d_gates = moeq.combine_grad(base.cuda(), pos.cuda(), gates=gates.cuda(), rows=rows.cuda(), out=rows.cuda())
    ref_r, ref_g, mag = products.combine_grad(_np(base), pos.numpy(), gates, _np(rows), P, _np(rows))
    _close(d_rows, ref_r, np.abs(ref_r), 1, "d_rows")
    _close(d_gates, ref_g, mag, N + 1, "d_gates")


def test_gradients_of_rows_beyond_32_bit_offsets():
    """Whole numbers, whose sums are exact: rows read and gradients written
    beyond 2^32 bytes and elements of the base, the rows left as they were."""
    from bit_quantized_moe_token_amd import moeq
    N, P = 1 << 20, 4200                              # 8.8 GB each
    g = torch.Generator().manual_seed(1)
    rows = torch.zeros((P, N), dtype=F16, device="cuda")
    out = torch.zeros_like(rows)
    pos = torch.tensor([P - 1, 3, 4097, P - 2], dtype=torch.int32)
    vals, dy = torch.randint(-8, 9, (4, N), generator=g).half(), torch.randint(-4, 5, (2, N), generator=g).half()
    rows[pos.long().cuda()] = vals.cuda()
    gates = torch.tensor([[0.5, 0.25], [1.0, 2.0]])
    d, dg = moeq.combine_grad(dy.cuda(), pos.cuda(), gates=gates.cuda(), rows=rows, out=out)
    for p in range(4):
        assert torch.equal(d[int(pos[p])].cpu(), (gates.view(-1)[p] * dy[p // 2].float()).half())
        assert float(dg.view(-1)[p]) == float(dy[p // 2].double() @ vals[p].double())
        assert torch.equal(rows[int(pos[p])].cpu(), vals[p])
    d[pos.long().cuda()] = 0
    assert not d.any()                                # nothing anywhere else


def test_refusals():
    from bit_quantized_moe_token_amd import moeq
    rows, pos, g = torch.ones(8, 16).half().cuda(), torch.arange(8, dtype=torch.int32).cuda(), torch.ones(4, 2).cuda()
    for a, kw, e in (((rows.cpu(), pos), dict(gates=g), TypeError), ((rows, pos.long()), dict(gates=g), TypeError),
                     ((rows, pos), dict(), ValueError), ((rows, pos[:7]), dict(gates=g), ValueError),
                     ((rows, pos), dict(gates=g, k=3), ValueError), ((rows, pos), dict(k=3), ValueError),
                     ((rows, pos), dict(k=0), ValueError), ((rows, pos), dict(gates=g.half()), TypeError),
                     ((rows, pos), dict(gates=g.T), ValueError), ((rows.T, pos), dict(gates=g), ValueError),
                     ((rows, pos), dict(gates=g, base=rows), ValueError),
                     ((rows, pos), dict(gates=g, out=torch.ones(4, 16).bfloat16().cuda()), TypeError),
                     ((rows, pos), dict(gates=g, out=torch.ones(4, 15).half().cuda()), ValueError)):
        with pytest.raises(e):
            moeq.combine(*a, **kw)
    with pytest.raises(moeq.MoeqError):
        moeq.combine(rows, pos, gates=g, out_dtype=BF16)
    with pytest.raises(moeq.MoeqError):
        moeq.combine(rows, pos, gates=g, out=torch.ones(1, 16).half().cuda().expand(4, 16))
    dy = torch.ones(4, 16).half().cuda()
    for a, kw, e in (((dy.cpu(), pos), dict(gates=g), TypeError), ((dy[:3], pos), dict(gates=g), ValueError),
                     ((dy, pos), dict(gates=g, rows=rows[:, :8]), ValueError),
                     ((dy, pos), dict(gates=g, rows=rows.bfloat16()), TypeError),
                     ((dy, pos), dict(gates=g, rows=rows, out=rows[:7]), ValueError),
                     ((dy, pos), dict(gates=g, rows=rows, out_dtype=F32), TypeError),
                     ((dy, pos), dict(gates=g, out_dtype=torch.float64), TypeError)):
        with pytest.raises(e):
            moeq.combine_grad(*a, **kw)


def test_no_slots_and_no_tokens_are_refused_as_arguments():
    from bit_quantized_moe_token_amd import moeq
    rows, none = torch.ones(8, 16).half().cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    for k in (0, -1):
        with pytest.raises(ValueError):
            moeq.combine(rows, none, k=k)
        with pytest.raises(ValueError):
            moeq.combine_grad(rows[:0], none, k=k)


def test_two_streams_and_captured_calls():
    from bit_quantized_moe_token_amd import moeq
    T, k, N = 500, 6, 1408
    sets = [(_rand((T * k, N), BF16, s).cuda(), _positions(T, k, T * k, s).cuda(), torch.rand(T, k).cuda(),
             _rand((T, N), BF16, s + 9).cuda()) for s in (0, 1)]

    def passes(rows, pos, gates, dy):
        return [moeq.combine(rows, pos, gates=gates, base=dy), *moeq.combine_grad(dy, pos, gates=gates, rows=rows)]

    ref = [[t.clone() for t in passes(*s)] for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for _ in range(3):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(passes(*s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, ref[i % 2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = passes(*sets[0])
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref[0]))
        assert all(torch.equal(a, b) for a, b in zip(passes(*sets[0]), ref[0]))
