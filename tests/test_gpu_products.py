"""Products of expert-sorted rows (16-bit, their gradients, 8-bit) against the
fp64 forms of oracle/products.py.

Tolerances, per element.  16-bit inputs multiply exactly in fp32, and a sum of
n terms in fp32 in any order, each step off by at most one unit in the last
place (2^-23 relative, which also covers a truncating adder), is off by at
most n 2^-23 times the sum of the terms' magnitudes; the result is rounded
once to the output's type (half a step, plus half the smallest subnormal).
8-bit: the integer sum is exact; its conversion and two scalings are three
fp32 roundings of 2^-24 each.
"""

import numpy as np
import pytest

from oracle import products

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}


def _np(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def _round_tol(ref, dtype):
    return np.abs(ref) * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def _check(got, ref, tol, what):
    got = _np(got)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} of the tolerance, first at "
                           f"{np.argwhere(bad)[0]}")


def _routing(rng, counts, k, T, before=0, behind=0):
    """Offsets and pairs of rows sorted by expert, `before` and `behind` rows
    outside every expert."""
    P = before + sum(counts) + behind
    off = np.concatenate([[0], np.cumsum(counts)]) + before
    pairs = rng.integers(0, T * k, size=P)
    return off.astype(np.int32), pairs.astype(np.int32)


def _rows(rng, shape, dtype, ld=None, lead=0, scale=1.0):
    """Random matrix (or matrices) as a view with row stride ld, `lead`
    elements into its storage; everything around the values is NaN."""
    rows, cols = int(np.prod(shape[:-1])), shape[-1]
    ld = ld or cols
    buf = torch.full((lead + rows * ld,), float("nan"), dtype=dtype, device="cuda")
    v = buf[lead:].view(*shape[:-1], ld)[..., :cols]
    v.copy_(torch.from_numpy(scale * rng.standard_normal(shape)).to(dtype).cuda())
    return v


# counts per expert, k, K, N: from one row to several tiles, odd and aligned widths
SHAPES = [
    ([1], 1, 1, 1),
    ([1], 1, 64, 16),
    ([0, 1, 0], 2, 65, 17),
    ([3, 0, 16, 17], 2, 128, 256),
    ([5, 1, 2], 3, 1000, 131),
    ([40, 0, 0, 7], 4, 192, 129),
    ([129, 64, 1], 2, 256, 384),
    ([300, 33], 1, 77, 260),
    ([257, 513, 3, 0], 2, 320, 520),
    ([0, 0], 2, 96, 40),
    ([2] * 70 + [0] * 9 + [31], 8, 136, 72),
    ([1] * 200 + [0] * 56, 2, 64, 64),
    ([700], 1, 1030, 258),
    ([33, 5], 2, 72, 2000),
    ([1100, 3, 900, 0], 2, 144, 6664),      # enough tiles for the largest ones
    ([9, 9, 9], 1, 40, 33),
    ([50, 0, 70, 33], 1, 2056, 2104),       # and in the matrices' gradient
    ([600, 2, 811], 2, 200, 6300),
    # each tile of the aligned and, at odd indices, of the unaligned path;
    # long rows and few tiles take longer rings
    ([90] * 15 + [91], 2, 144, 2500),
    ([90] * 15 + [91], 2, 135, 1001),
    ([50] * 16, 2, 144, 2500),
    ([50] * 16, 2, 133, 1003),
    ([90] * 16, 2, 2048, 1000),
    ([7, 0, 3], 1, 2100, 50),
    ([50] * 16, 2, 2048, 1000),
    ([3] * 5, 1, 77, 130),
    ([3, 9, 1], 2, 4096, 200),
    ([1, 2], 1, 19, 70),
    ([3] * 60, 1, 80, 600),
    ([20] * 40, 2, 99, 300),
    ([20] * 40, 2, 96, 300),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("trans", [False, True], ids=["fwd", "trans"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_grouped_gemm(i, trans, dtype):
    from bit_quantized_moe_token_amd import moeq
    counts, k, K, N = SHAPES[i]
    rng = np.random.default_rng(100 * i + 7 * trans)
    E, T = len(counts), max(1, sum(counts) // k)
    off, pairs = _routing(rng, counts, k, T, before=i % 3, behind=i % 2 * 5)
    # every second shape: strided rows at an odd start, NaN around them
    odd = i % 2
    x = _rows(rng, (T, K), dtype, ld=K + 3 * odd, lead=odd)
    w = _rows(rng, (E, K, N) if trans else (E, N, K), dtype, ld=(N if trans else K) + 5 * odd, lead=3 * odd)
    out_dtype = F32 if i % 4 >= 2 else dtype
    P = len(pairs)
    out = torch.full((P, N), 7.0, dtype=out_dtype, device="cuda")
    r = moeq.grouped_gemm(x, w, torch.from_numpy(off).cuda(), pairs=torch.from_numpy(pairs).cuda(), k=k, trans=trans,
                          out=out)
    assert r is out
    wn = _np(w).swapaxes(1, 2) if trans else _np(w)
    src = products.source_rows(P, T, pairs, k)
    seven, zero = np.full((P, N), 7.0), np.zeros((P, N))
    ref = products.grouped(_np(x), wn, off, src, seven)
    mag = products.grouped(np.abs(_np(x)), np.abs(wn), off, src, zero)
    _check(out, ref, K * 2.0 ** -23 * mag + _round_tol(ref, out_dtype), SHAPES[i])
    outside = np.ones(P, bool)
    outside[off[0]:off[-1]] = False
    assert np.all(_np(out)[outside] == 7.0)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_grouped_wgrad(i, dtype):
    from bit_quantized_moe_token_amd import moeq
    counts, k, K, N = SHAPES[i]
    rng = np.random.default_rng(1000 + i)
    E, T = len(counts), max(1, sum(counts) // k)
    off, pairs = _routing(rng, counts, k, T, before=i % 3, behind=i % 2 * 5)
    odd = i % 2
    P = len(pairs)
    x = _rows(rng, (T, K), dtype, ld=K + 3 * odd, lead=odd)
    dy = _rows(rng, (P, N), dtype, ld=N + 7 * odd, lead=odd)
    dy[: off[0]] = float("nan")
    dy[off[-1]:] = float("nan")
    out_dtype = dtype if i % 4 >= 2 else F32
    dw = moeq.grouped_wgrad(dy, x, torch.from_numpy(off).cuda(), pairs=torch.from_numpy(pairs).cuda(), k=k,
                            out_dtype=out_dtype)
    src = products.source_rows(P, T, pairs, k)
    ref = products.wgrad(_np(dy), _np(x), off, src)
    mag = products.wgrad(np.abs(_np(dy)), np.abs(_np(x)), off, src)
    n = np.asarray(counts, dtype=np.float64)[:, None, None]
    _check(dw, ref, n * 2.0 ** -23 * mag + _round_tol(ref, out_dtype), SHAPES[i])


@pytest.mark.parametrize("E,K,N,ld", [(200, 264, 392, 0), (256, 40, 300, 0), (3, 2600, 1112, 0), (90, 130, 1200, 1), (1, 2200, 2200, 0)])
def test_wgrad_of_uneven_experts(E, K, N, ld):
    """Experts in every class of rows, more than a lane's worth of them, more
    tiles than a round of runs, more columns of tiles than a band."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(E)
    counts = rng.choice([0, 1, 7, 40, 130, 500], size=E, p=[0.2, 0.2, 0.2, 0.2, 0.15, 0.05]) if E > 3 else [330, 0, 21][:E]
    off, pairs = _routing(rng, counts, 2, 300, before=3, behind=2)
    x = _rows(rng, (300, K), BF16, ld=K + ld)
    dy = _rows(rng, (len(pairs), N), BF16, ld=N + ld)
    dw = moeq.grouped_wgrad(dy, x, torch.from_numpy(off).cuda(), pairs=torch.from_numpy(pairs).cuda(), k=2, out_dtype=F32)
    src = products.source_rows(len(pairs), 300, pairs, 2)
    ref = products.wgrad(_np(dy), _np(x), off, src)
    mag = products.wgrad(np.abs(_np(dy)), np.abs(_np(x)), off, src)
    n = np.asarray(counts, dtype=np.float64)[:, None, None]
    _check(dw, ref, n * 2.0 ** -23 * mag + _round_tol(ref, F32), (E, K, N))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("counts,K,N", [([70, 0, 9], 72, 133), ([90] * 16, 88, 1003), ([700, 300], 104, 6661), ([3], 8, 1)])
def test_padded_rows(counts, K, N, dtype):
    """Rows that start at multiples of 16 bytes and end within one, NaN
    between them, in a tensor that ends with its last row."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(N)
    E, P = len(counts), sum(counts)
    pad = lambda n: (n + 7) // 8 * 8 + 8

    def rows(*shape):
        ld, count = pad(shape[-1]), int(np.prod(shape[:-1]))
        buf = torch.full(((count - 1) * ld + shape[-1],), float("nan"), dtype=dtype, device="cuda")
        strides = (shape[-2] * ld, ld, 1) if len(shape) == 3 else (ld, 1)
        return buf.as_strided(shape, strides).copy_(torch.from_numpy(rng.standard_normal(shape)).to(dtype))

    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    src = np.arange(P)
    zero = np.zeros((P, N))
    # the rows' gradient: w [E, K, N] with N no multiple of 8
    x, w = rows(P, K), rows(E, K, N)
    y = moeq.grouped_gemm(x, w, off, trans=True)
    wn = _np(w).swapaxes(1, 2)
    ref = products.grouped(_np(x), wn, off.cpu().numpy(), src, zero)
    mag = products.grouped(np.abs(_np(x)), np.abs(wn), off.cpu().numpy(), src, zero)
    _check(y, ref, K * 2.0 ** -23 * mag + _round_tol(ref, dtype), "trans")
    # the matrices' gradient: dy [P, N]
    dy = rows(P, N)
    for a, b, what in ((dy, x, "wgrad"), (x, dy, "wgrad, the other way")):
        dw = moeq.grouped_wgrad(a, b, off)
        ref = products.wgrad(_np(a), _np(b), off.cpu().numpy(), src)
        mag = products.wgrad(np.abs(_np(a)), np.abs(_np(b)), off.cpu().numpy(), src)
        n = np.asarray(counts, dtype=np.float64)[:, None, None]
        _check(dw, ref, n * 2.0 ** -23 * mag + _round_tol(ref, F32), what)


def test_grouped_without_pairs_and_bad_pairs():
    """Without pairs row r reads row r; a pair outside the source rows reads
    zeros; offsets outside [0, P] count as its ends."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(3)
    x, w = _rows(rng, (50, 72), F16), _rows(rng, (2, 24, 72), F16)
    off = torch.tensor([-4, 20, 90], dtype=torch.int32).cuda()
    y = moeq.grouped_gemm(x, w, off, out_dtype=F32)
    for wild in ([0, 50, 0], [50, 0, 50], [2147483647, -2147483648, 2147483647]):     # nothing to hold them to but bounds
        moeq.grouped_gemm(x, w, torch.tensor(wild, dtype=torch.int32).cuda())
        moeq.grouped_wgrad(x, x, torch.tensor(wild, dtype=torch.int32).cuda())
    ref = products.grouped(_np(x), _np(w), [0, 20, 50], np.arange(50), np.zeros((50, 24)))
    mag = products.grouped(np.abs(_np(x)), np.abs(_np(w)), [0, 20, 50], np.arange(50), np.zeros((50, 24)))
    _check(y, ref, 72 * 2.0 ** -23 * mag + _round_tol(ref, F32), "no pairs")
    pairs = np.arange(50, dtype=np.int32) * 2
    pairs[[3, 30]] = [100, -1]
    y = moeq.grouped_gemm(x, w, off, pairs=torch.from_numpy(pairs).cuda(), k=2, out_dtype=F32)
    ref[[3, 30]] = 0
    _check(y, ref, 72 * 2.0 ** -23 * mag + _round_tol(ref, F32), "bad pairs")
    dy = _rows(rng, (50, 24), F16)
    dw = moeq.grouped_wgrad(dy, x, off, pairs=torch.from_numpy(pairs).cuda(), k=2)
    src = products.source_rows(50, 50, pairs, 2)
    ref = products.wgrad(_np(dy), _np(x), [0, 20, 50], src)
    mag = products.wgrad(np.abs(_np(dy)), np.abs(_np(x)), [0, 20, 50], src)
    _check(dw, ref, 30 * 2.0 ** -23 * mag + _round_tol(ref, F32), "bad pairs, wgrad")


def test_infinities_stay_in_their_rows():
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(4)
    x, w = _rows(rng, (40, 64), BF16), _rows(rng, (1, 48, 64), BF16)
    x[5, 3], x[17, 0] = float("inf"), float("nan")
    y = _np(moeq.grouped_gemm(x, w, torch.tensor([0, 40], dtype=torch.int32).cuda()))
    hit = ~np.isfinite(y).all(1)
    assert set(np.argwhere(hit)[:, 0]) == {5, 17} and np.isnan(y[17]).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 65), (257, 130), (2, 20000), (9, 7)])
def test_quantize_i8(rows, cols, dtype):
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(rows * 31 + cols)
    x = _rows(rng, (rows, cols), dtype, ld=cols + rows % 2 * 3, lead=rows % 2)
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-4
    if rows > 4:
        x[3, cols // 2], x[4, 0] = float("inf"), float("nan")
    if dtype != F16 and rows > 5:
        x[5] = 2.0 ** -126     # its scale would be subnormal
        x[6] = 2.0 ** -118
    q, s = moeq.quantize_i8(x)
    with np.errstate(invalid="ignore"):
        qr, sr = products.code_i8(x.to(torch.float32).cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), qr)
    assert np.array_equal(s.cpu().numpy(), sr, equal_nan=True)


def test_codes_of_halves():
    """Rows whose scale is a small integer: values half way between two codes
    go to the even one."""
    from bit_quantized_moe_token_amd import moeq
    s = torch.arange(9, 17, dtype=torch.float32)[:, None]
    x = (torch.arange(-127, 128, dtype=torch.float32)[None] / 2 * s).cuda()
    x[:, 0] = 127 * s[:, 0].cuda()
    for dtype in (F16, BF16, F32):
        xr = x.to(dtype)
        q, scale = moeq.quantize_i8(xr)
        qr, sr = products.code_i8(xr.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(scale.cpu().numpy(), sr)
        # fp16 and fp32 hold these rows exactly: the scale is s, and the
        # quotients are exact.  (bf16 rounds 127 s, then s, so that quotients
        # of x / scale in more bits are no halves any more: the fp32 quotient
        # above is the definition.)
        if dtype != BF16:
            assert torch.equal(scale.cpu(), s[:, 0])
            assert torch.equal(q.double(), torch.round(x.double() / s.double().cuda()))


I8_SHAPES = SHAPES + [([201], 1, 1530, 1111), ([16], 1, 4096, 64), ([64], 1, 130, 300), ([4], 1, 16384, 32),
                      ([0, 1], 1, 33, 5), ([90] * 16, 2, 4096, 1000), ([1], 1, 20001, 40), ([50] * 16, 2, 4096, 1000)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("i", range(len(I8_SHAPES)))
def test_i8(i, dtype):
    """gemm_i8 against the exact integer product, and linear_i8 equal to
    quantize_i8 followed by gemm_i8, bit for bit."""
    from bit_quantized_moe_token_amd import moeq
    counts, k, K, N = I8_SHAPES[i]
    rng = np.random.default_rng(2000 + i)
    dense = len(counts) == 1 and i % 2 == 0
    E, T = len(counts), max(1, sum(counts) // k)
    off, pairs = _routing(rng, counts, k, T, before=0 if dense else i % 3, behind=0 if dense else i % 2 * 5)
    odd = i % 2
    x = _rows(rng, (T, K), dtype, ld=K + 3 * odd, lead=odd)
    if T > 3:
        x[1], x[2, 0] = 0, float("nan")
    wq = torch.from_numpy(rng.integers(-127, 128, size=(E, N, K + 3 * odd)).astype(np.int8)).cuda()[:, :, :K]
    sw = torch.from_numpy(rng.uniform(0.5, 1.5, size=(E, N)).astype(np.float32) / 64).cuda()
    P = T if dense else len(pairs)
    kw = {} if dense else dict(offsets=torch.from_numpy(off).cuda(), pairs=torch.from_numpy(pairs).cuda(), k=k)
    if dense:
        off, wq, sw = np.array([0, T]), wq[0], sw[0]
        src = np.arange(T)
    else:
        src = products.source_rows(P, T, pairs, k)
    out = torch.full((P, N), 7.0, dtype=dtype, device="cuda")
    xq, sx = moeq.quantize_i8(x)
    got = moeq.gemm_i8(xq, sx, wq, sw, out=out, **kw)
    ints = products.grouped(xq.cpu().numpy(), wq.cpu().numpy().reshape(E, N, K), off, src, np.zeros((P, N)))
    s = products.gather(sx.cpu().numpy()[:, None], src)
    ref = np.full((P, N), 7.0)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        ref[rows] = ints[rows] * s[rows] * sw.cpu().numpy().reshape(E, N)[e]
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(_np(got)), nan)
    _check(torch.nan_to_num(got), np.nan_to_num(ref), 3 * 2.0 ** -24 * np.abs(np.nan_to_num(ref)) * (1 + 2.0 ** -8) +
           _round_tol(np.nan_to_num(ref), dtype) * (1 + 2.0 ** -8), I8_SHAPES[i])
    out2 = torch.full((P, N), 7.0, dtype=dtype, device="cuda")
    moeq.linear_i8(x, wq, sw, out=out2, **kw)
    assert torch.equal(torch.nan_to_num(out2), torch.nan_to_num(got))


def test_i8_sum_is_exact_at_its_longest():
    """The integer sum of 131071 products of -128 x -128 and of 127 x -127 is
    exact (longer rows are refused)."""
    from bit_quantized_moe_token_amd import moeq
    K = 131071
    xq = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((17, K), -128, dtype=torch.int8, device="cuda")
    xq[1], wq[1] = 127, -127
    one, ones = torch.ones(2, device="cuda"), torch.ones(17, device="cuda")
    y = moeq.gemm_i8(xq, one, wq, ones, out_dtype=F32)
    want = torch.tensor([-128, 127], dtype=torch.float64)[:, None] * wq[:, 0].cpu().double()[None] * K
    assert torch.equal(y.cpu(), want.float())


def test_subnormal_inputs():
    """Subnormal fp16 and bf16 values keep their value in the products."""
    from bit_quantized_moe_token_amd import moeq
    off = torch.tensor([0, 4], dtype=torch.int32).cuda()
    for dtype, small in ((F16, 2.0 ** -24), (BF16, 2.0 ** -130)):
        x = (torch.arange(1, 5, device="cuda")[:, None].double() * small).to(dtype).expand(4, 64).contiguous()
        w = torch.full((1, 32, 64), 2.0 ** 14, dtype=dtype, device="cuda")
        y = moeq.grouped_gemm(x, w, off, out_dtype=F32)
        assert torch.equal(y.double(), (x[:, :1].double() * 2.0 ** 20).expand(4, 32))
        dw = moeq.grouped_wgrad(w[0].T[:4].contiguous(), x, off)
        assert torch.equal(dw.double(), x.double().sum(0).expand(1, 32, 64) * 2.0 ** 14)


def test_offsets_beyond_32_bits():
    """Source rows, matrices and outputs that lie more than 2^32 bytes into
    their tensors."""
    from bit_quantized_moe_token_amd import moeq
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").half()

    def check(y, x, w):
        ref, mag = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
        _check(y, ref.cpu().numpy(), (x.shape[1] * 2.0 ** -23 * mag).cpu().numpy() + _round_tol(ref.cpu().numpy(), F16), "far")

    T, K, N = 1100000, 2048, 96                      # x: 4.5 GB
    x = torch.zeros(T, K, dtype=F16, device="cuda")
    rows = torch.tensor([0, 5, T // 2, T - 2, T - 1], device="cuda")
    x[rows] = rand(5, K)
    w = rand(1, N, K)
    off = torch.tensor([0, 5], dtype=torch.int32).cuda()
    check(moeq.grouped_gemm(x, w, off, pairs=rows.int(), k=1), x[rows], w[0])
    dy = rand(5, N)
    dw = moeq.grouped_wgrad(dy, x, off, pairs=rows.int(), k=1)
    ref = dy.double().T @ x[rows].double()
    _check(dw[0], ref.cpu().numpy(), (5 * 2.0 ** -23 * (dy.double().abs().T @ x[rows].double().abs())).cpu().numpy() +
           _round_tol(ref.cpu().numpy(), F32), "far wgrad")
    q, s = moeq.quantize_i8(x)
    qr, sr = products.code_i8(x[rows].float().cpu().numpy())
    assert np.array_equal(q[rows].cpu().numpy(), qr) and np.array_equal(s[rows].cpu().numpy(), sr)
    del x, q, s
    E, N, K = 5, 65536, 8192                         # w: 5.4 GB
    w = torch.zeros(E, N, K, dtype=F16, device="cuda")
    w[E - 1, N - 300:] = rand(300, K)
    x = rand(3, K)
    y = moeq.grouped_gemm(x, w, torch.tensor([0, 0, 0, 0, 0, 3], dtype=torch.int32).cuda())
    check(y[:, N - 300:], x, w[E - 1, N - 300:])
    assert not y[:, :N - 300].any()
    del w
    P, N, K = 300000, 8192, 16                       # y: 4.9 GB
    x, w = rand(P, K), rand(1, N, K)
    y = moeq.grouped_gemm(x, w, torch.tensor([0, P], dtype=torch.int32).cuda())
    check(y[P - 40:, 4000:4100], x[P - 40:], w[0, 4000:4100])
    check(y[:40, 4000:4100], x[:40], w[0, 4000:4100])


def test_graph_stream_and_repeat():
    """A captured pass of all products, replayed with eager work between the
    replays, gives the eager results bit for bit; so does a call on another
    stream, and a repeated call."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(9)
    counts, k, K, N = [150, 0, 9, 41], 2, 256, 384
    off, pairs = _routing(rng, counts, k, 100)
    off, pairs = torch.from_numpy(off).cuda(), torch.from_numpy(pairs).cuda()
    x, w = _rows(rng, (100, K), BF16), _rows(rng, (4, N, K), BF16)
    wq, sw = moeq.quantize_i8(w)

    def step():
        y = moeq.grouped_gemm(x, w, off, pairs=pairs, k=k)
        return y, moeq.grouped_gemm(y, w, off, trans=True), moeq.grouped_wgrad(y, x, off, pairs=pairs, k=k), \
            moeq.linear_i8(x, wq, sw, offsets=off, pairs=pairs, k=k)

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
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        assert all(torch.equal(a, b) for a, b in zip(step(), eager))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_refusals():
    from bit_quantized_moe_token_amd import moeq
    x, w = torch.zeros(4, 64, dtype=F16, device="cuda"), torch.zeros(2, 32, 64, dtype=F16, device="cuda")
    off, pairs = torch.tensor([0, 2, 4], dtype=torch.int32).cuda(), torch.zeros(4, dtype=torch.int32).cuda()
    ok = moeq.grouped_gemm(x, w, off, pairs=pairs, k=1)
    assert ok.shape == (4, 32)
    for bad, err in (((x.cpu(), w, off), TypeError), ((x.float(), w, off), TypeError), ((x, w.bfloat16(), off), TypeError),
                     ((x, w[0], off), ValueError), ((x[:, :63], w, off), ValueError), ((x.T, w, off), ValueError),
                     ((x, w, off[:2]), ValueError), ((x, w, off.long()), TypeError), ((x, w, None), ValueError)):
        with pytest.raises(err):
            moeq.grouped_gemm(*bad)
    with pytest.raises(TypeError):
        moeq.grouped_gemm(x, w, off, out=torch.zeros(4, 32, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        moeq.grouped_gemm(x, w, off, out=torch.zeros(4, 31, dtype=F16, device="cuda"))
    with pytest.raises(ValueError):
        moeq.grouped_gemm(x, w, off, trans=True)                     # 64 columns against 32
    with pytest.raises(moeq.MoeqError):
        moeq.grouped_gemm(x, w, off, pairs=pairs, k=0)
    with pytest.raises(moeq.MoeqError):
        moeq.grouped_gemm(x[:1].expand(4, 64), w, off)               # rows that lie on each other
    with pytest.raises(ValueError):
        moeq.grouped_wgrad(x, x, off, pairs=pairs[:3])
    with pytest.raises(moeq.MoeqError):
        moeq.grouped_wgrad(x, x, off, out=torch.zeros(1, 64, 64, device="cuda").expand(2, 64, 64))
    wq, sw = torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.ones(32, device="cuda")
    for bad, err in (((x, wq.float(), sw), TypeError), ((x, wq[:, :63], sw), ValueError), ((x, wq, sw[:31]), ValueError),
                     ((x, wq, sw.half()), TypeError), ((x.double(), wq, sw), TypeError)):
        with pytest.raises(err):
            moeq.linear_i8(*bad)
    with pytest.raises(moeq.MoeqError) as e:
        moeq.linear_i8(x, wq, sw, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3


def test_equal_inputs_and_shared_matrices():
    """The same source row at several places gives equal rows; experts may
    share one matrix (stride 0); outputs may be a view with gaps."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(12)
    x, w = _rows(rng, (3, 80), BF16), _rows(rng, (1, 48, 80), BF16)
    off = torch.tensor([0, 70, 70, 200], dtype=torch.int32).cuda()
    pairs = torch.from_numpy((np.arange(200) % 3 * 2).astype(np.int32)).cuda()
    buf = torch.full((200, 61), 5.0, dtype=BF16, device="cuda")
    y = moeq.grouped_gemm(x, w.expand(3, 48, 80), off, pairs=pairs, k=2, out=buf[:, :48])
    one = moeq.grouped_gemm(x, w, torch.tensor([0, 3], dtype=torch.int32).cuda())
    assert torch.equal(y, one[torch.arange(200, device="cuda") % 3])
    assert bool((buf[:, 48:] == 5).all())


def test_two_streams_and_two_graphs():
    """Two captured passes and eager ones on two streams, each with outputs
    and workspaces of its own, do not disturb each other."""
    from bit_quantized_moe_token_amd import moeq
    rng = np.random.default_rng(13)
    passes = []
    for n in (300, 40):
        off, pairs = _routing(rng, [n, 5, n // 2], 2, 64)
        x, w = _rows(rng, (64, 512), F16), _rows(rng, (3, 256, 512), F16)
        wq, sw = moeq.quantize_i8(w)
        passes.append((torch.from_numpy(off).cuda(), torch.from_numpy(pairs).cuda(), x, w, wq, sw))

    def step(p):
        off, pairs, x, w, wq, sw = p
        y = moeq.grouped_gemm(x, w, off, pairs=pairs, k=2)
        return y, moeq.linear_i8(x, wq, sw, offsets=off, pairs=pairs, k=2), moeq.grouped_wgrad(y, x, off, pairs=pairs, k=2)

    eager = [[t.clone() for t in step(p)] for p in passes]
    graphs, outs = [], []
    for p in passes:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(p))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        live = []
        for g, s, p in zip(graphs, streams, passes):
            with torch.cuda.stream(s):
                g.replay()
                live.append(step(p))
        torch.cuda.synchronize()
        for o, l, e in zip(outs, live, eager):
            assert all(torch.equal(a, b) for a, b in zip(o, e))
            assert all(torch.equal(a, b) for a, b in zip(l, e))
