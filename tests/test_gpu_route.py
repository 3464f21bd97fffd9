"""GPU parity of routing and the counting sort: ids, offsets, sorted pairs and
their inverse bit-exact against the oracle; gates within 2e-6."""

import numpy as np
import pytest

from oracle import forward
from synth import configs, gen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _route(logits, k):
    from bit_quantized_moe_token_amd import moeq
    rt = moeq.route(torch.from_numpy(logits).cuda(), k)
    torch.cuda.synchronize()
    return rt


def _check(logits, k):
    rt = _route(logits, k)
    ref = forward.route(logits, k)
    T = logits.shape[0]
    assert np.array_equal(rt.offsets.cpu().numpy(), ref["offsets"])
    if T == 0:
        return
    assert np.array_equal(rt.ids.cpu().numpy(), ref["ids"])
    assert np.array_equal(rt.sorted_pairs.cpu().numpy(), ref["sorted_pairs"])
    assert np.array_equal(rt.pair_pos.cpu().numpy(), ref["pair_pos"])
    g = rt.gates.cpu().numpy().astype(np.float64)
    assert np.max(np.abs(g - ref["gates"])) <= 2e-6
    # the kernel's softmax denominator is an fp32 sum of k terms, so the k
    # fp32 gates sum to 1 within about k units of 2^-24 (k + 4 ulp of 1 here)
    assert np.max(np.abs(g.sum(1) - 1)) <= max(2e-6, (k + 4) * 2.0 ** -23)


@pytest.mark.parametrize("name", ["tiny", "decode", "prefill", "finegrained", "bitplane"])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_route_configs(name, seed):
    cfg = configs.get(name)
    _check(gen.gen_logits(cfg, seed), cfg["k"])


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 8, 8), (5, 3, 1), (333, 256, 7), (70, 64, 64),
                                   (2000, 5, 2), (1030, 128, 8), (4096, 2, 2), (64, 8, 2), (65, 256, 256),
                                   (129, 7, 3), (16, 256, 256), (17, 8, 2), (16, 8, 2)])
def test_route_shapes_and_ties(T, E, k):
    rng = np.random.default_rng(T + E + k)
    logits = (rng.integers(-2, 3, size=(T, E)) * 0.25).astype(np.float32)   # many ties
    _check(logits, k)
    _check(rng.standard_normal((T, E)).astype(np.float32), k)


@pytest.mark.parametrize("T,E,k", [(4097, 8, 2), (8192, 256, 8), (5000, 64, 6)])
def test_route_long_batches(T, E, k):
    """Beyond 4096 tokens the sort counts through a workspace (per-segment
    histograms, one scan over the segments): bit-exact against the oracle
    on tied and untied logits, with a ragged last segment (4097, 5000)."""
    from bit_quantized_moe_token_amd import moeq
    rt = moeq.RoutingOut(T, E, k, "cuda")
    assert rt.ws_bytes == -(-T // 64) * E * 4
    rng = np.random.default_rng(T + E)
    _check((rng.integers(-2, 3, size=(T, E)) * 0.25).astype(np.float32), k)
    _check(rng.standard_normal((T, E)).astype(np.float32), k)


@pytest.mark.parametrize("T,E,k", [(8193, 7, 2), (8193, 64, 6), (10241, 256, 8), (20001, 256, 2), (32768, 128, 8),
                                   (65536, 64, 3)])
def test_route_batches_of_many_segments(T, E, k):
    """More than 128 segments: each of the scan's parts has more of them than
    it keeps in registers, with ragged last segments and parts."""
    rng = np.random.default_rng(T + E)
    _check((rng.integers(-2, 3, size=(T, E)) * 0.25).astype(np.float32), k)
    _check(rng.standard_normal((T, E)).astype(np.float32), k)


def test_route_deterministic():
    cfg = configs.get("prefill")
    logits = gen.gen_logits(cfg, 0)
    a = _route(logits, 2)
    b = _route(logits, 2)
    for f in ("ids", "gates", "offsets", "sorted_pairs", "pair_pos"):
        assert torch.equal(getattr(a, f), getattr(b, f))


# ---- routing mass (per-expert gate-weighted usage and its buckets)

@pytest.mark.parametrize("name", ["tiny", "decode", "prefill", "finegrained", "bitplane"])
def test_route_mass(name):
    from bit_quantized_moe_token_amd import moeq
    cfg = configs.get(name)
    logits = gen.gen_logits(cfg, 0)
    rt = _route(logits, cfg["k"])
    ref = forward.route(logits, cfg["k"])
    m_ref = forward.routing_mass(ref["ids"], ref["gates"], cfg["E"])
    # edges around the typical mass, including one at an exactly representable value
    mean = cfg["T"] * cfg["k"] / cfg["E"] / cfg["k"]
    edges = [0.0, 0.5 * mean, mean, 2.0 * mean, 4.0]
    edges = sorted(edges)
    mass, bucket = moeq.route_mass(rt, edges)
    torch.cuda.synchronize()
    m = mass.cpu().numpy().astype(np.float64)
    # fp32 sums of at most T gates in [0, 1]
    assert np.all(np.abs(m - m_ref) <= 1e-5 * np.maximum(1.0, m_ref)), np.max(np.abs(m - m_ref))
    assert abs(m.sum() - cfg["T"]) <= 1e-5 * cfg["T"]
    # the bucket decision is taken on the kernel's fp32 mass
    b_host = forward.mass_bucket(mass.cpu().numpy(), np.asarray(edges, dtype=np.float32))
    assert np.array_equal(bucket.cpu().numpy(), b_host)
    far = np.min(np.abs(m_ref[:, None] - np.asarray(edges)[None, :]), axis=1) > 1e-3
    assert np.array_equal(bucket.cpu().numpy()[far], forward.mass_bucket(m_ref, edges)[far])
    mass2, _ = moeq.route_mass(rt)
    assert torch.equal(mass, mass2)                     # deterministic; no buckets requested


def test_route_mass_validation():
    from bit_quantized_moe_token_amd import moeq
    rt = _route(np.zeros((4, 8), dtype=np.float32), 2)
    with pytest.raises(moeq.MoeqError):
        moeq.route_mass(rt, [2.0, 1.0])                  # not ascending
    with pytest.raises(moeq.MoeqError):
        moeq.route_mass(rt, list(range(9)))              # too many edges
