"""Attention over the whole range of what a cache and its queries may hold: value vectors of zeros and of very different
sizes beside each other, single tokens that hold most of the weight, small elements beside large ones, infinities. All
rows attend over one long sequence, so that every CTA sees most of it in one run of tiles."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_bounds as ab
import attention_ref as ref
from test_attention_gpu import Rows

pytestmark = pytest.mark.gpu

DEV = "cuda"
ROWS = 160  # at least one row a CTA


def _sink(rng, dtype, n, weight, amplitude, sink_value, heads=16, at=0):
    """A sequence of n tokens with values of about `amplitude`, whose token `at` draws about `weight` of the softmax and
    has values of size `sink_value`."""
    cache = ref.Cache(rng, 1, 128, 64, dtype, [n])
    k = rng.standard_normal((n, 1, 128)).astype(np.float32)
    k[:, 0, 0] = 0
    k[at] = 0
    k[at, 0, 0] = (np.log(n) + 1.1 + np.log(weight / (1 - weight))) * np.sqrt(128) / 8
    v = (rng.standard_normal((n, 1, 128)) * amplitude).astype(np.float32)
    v[at] = rng.standard_normal((1, 128)) * sink_value
    ab.put(cache, 0, np.arange(n), 0, k)
    ab.put(cache, 0, np.arange(n), 1, v)
    rows = Rows(rng, cache, heads, [0] * ROWS)
    q = rows.q.clone()
    q[:, :, 0] = 8
    _queries(rows, q)
    return rows


def _queries(rows, q):
    rows.q = q
    rows.q_dev = q.to(DEV)


def _check(rows, positions, which=(0, 77, ROWS - 1), absolute=0.0):
    k, v = rows.cache.tokens(0, positions)
    for r in which:
        ab.check(rows.dev["out"][r], rows.dev["lse"][r], rows.q[r].to(torch.float64).numpy(), k, v, rows.scale,
                 f"row {r}", absolute)


@pytest.mark.parametrize("n,weight,amplitude,sink_value", [
    (2048, 0.3, 1.0, 0.0), (2048, 0.5, 1.0, 0.0), (2048, 0.9, 1.0, 0.0), (32768, 0.3, 1.0, 0.0),  # a token of zeros
    (2048, 0.5, 1e-3, 0.0), (2048, 0.5, 1e-9, 0.0), (2048, 0.01, 1e-6, 0.0),
    (2048, 0.5, 1.0, 1.0), (131072, 0.5, 1.0, 1.0), (131072, 0.9, 1.0, 1.0),                      # before a long tail
    (2048, 0.5, 1.0, 1e-6), (2048, 1e-5, 1e-4, 1.0), (2048, 0.9, 1e20, 1e25),
])
@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_one_token_that_holds_much_of_the_weight(dtype, n, weight, amplitude, sink_value):
    rng = np.random.Generator(np.random.PCG64(n + int(weight * 100)))
    rows = _sink(rng, dtype, n, weight, amplitude, sink_value, heads=16 if n < 10000 else 3)
    assert rows.call(row_ke=torch.full((ROWS,), n, dtype=torch.int32, device=DEV)) == 0
    _check(rows, np.arange(n), (0, ROWS - 1) if n < 10000 else (77,))


@pytest.mark.parametrize("sink_value", [0.0, 1.0])
@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_a_selected_token_that_holds_much_of_the_weight(dtype, sink_value):
    rng = np.random.Generator(np.random.PCG64(12))
    rows = _sink(rng, dtype, 5000, 0.5, 0.01, sink_value, at=4321)
    ids = np.stack([np.r_[rng.permutation(4000)[:2000], -1, 4321] for _ in range(ROWS)]).astype(np.int32)
    for i in ids:
        rng.shuffle(i)
    assert rows.call(token_ids=torch.from_numpy(ids).to(DEV)) == 0
    for r in (0, 77, ROWS - 1):
        _check(rows, ids[r][ids[r] >= 0], [r])


@pytest.mark.parametrize("n", [1, 700])
def test_a_value_vector_below_the_reciprocal_range(n):
    """A value scale whose reciprocal is past fp32. The absolute term: a weight times such a scale is below the normal
    range (2^-126), times a code of at most 448."""
    rng = np.random.Generator(np.random.PCG64(n))
    cache = ref.Cache(rng, 1, 128, 64, "e4m3", [n])
    ab.put(cache, 0, [n // 2], 1, (rng.standard_normal((1, 1, 128)) * 1e-37).astype(np.float32))
    assert 0 < float(cache.scales[cache.table[0][n // 2 // 64], 1, 0, n // 2 % 64]) < 2.0 ** -129
    for strength in (0.0, 100.0):  # as heavy as any, and of no weight at all
        ab.put(cache, 0, [n // 2], 0, np.full((1, 1, 128), -strength, np.float32))
        rows = Rows(rng, cache, 16, [0] * ROWS)
        _queries(rows, rows.q.abs())
        assert rows.call(row_ke=torch.full((ROWS,), n, dtype=torch.int32, device=DEV)) == 0
        _check(rows, np.arange(n), absolute=2.0 ** -117)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_small_query_elements_beside_a_large_one(dtype):
    """The scores come from elements far below the head's largest, which meets keys of zero."""
    rng = np.random.Generator(np.random.PCG64(41))
    n = 1000
    cache = ref.Cache(rng, 1, 128, 64, dtype, [n])
    k = rng.standard_normal((n, 1, 128)).astype(np.float32)
    k[:, :, 9] = 0
    ab.put(cache, 0, np.arange(n), 0, k)
    rows = Rows(rng, cache, 16, [0] * ROWS)
    q = rows.q.clone()
    q[:, :, 9] = 2.0 ** torch.linspace(0, 40, 16)
    _queries(rows, q)
    assert rows.call(row_ke=torch.full((ROWS,), n, dtype=torch.int32, device=DEV)) == 0
    _check(rows, np.arange(n))


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_queries_that_are_not_finite(dtype, bad):
    """An infinite element makes scores of both infinities, and the head's result is NaN; other heads keep theirs."""
    rng = np.random.Generator(np.random.PCG64(42))
    n = 300
    cache = ref.Cache(rng, 1, 64, 16, dtype, [n])
    rows = Rows(rng, cache, 20, [0] * ROWS)
    clean = rows.q.clone()
    q = clean.clone()
    q[:, 3, 7] = bad
    rows.q_dev = q.to(DEV)
    assert rows.call(row_ke=torch.full((ROWS,), n, dtype=torch.int32, device=DEV)) == 0
    out = rows.dev["out"]
    assert bool(torch.isnan(out[:, 3]).all())
    keep = [h for h in range(20) if h != 3]
    k, v = cache.tokens(0, np.arange(n))
    for r in (0, ROWS - 1):
        ab.check(out[r, keep], rows.dev["lse"][r, keep], clean[r, keep].to(torch.float64).numpy(), k, v, rows.scale)


@pytest.mark.parametrize("n", [1, 300])
def test_values_that_are_infinite(n):
    """An infinite value of a token with any weight makes its element of the result infinite, and no other."""
    rng = np.random.Generator(np.random.PCG64(43 + n))
    cache = ref.Cache(rng, 1, 128, 64, "bf16", [n])
    at = n // 2
    v = rng.standard_normal((1, 1, 128)).astype(np.float32)
    v[0, 0, [5, 64]] = np.inf
    v[0, 0, 77] = -np.inf
    ab.put(cache, 0, [at], 1, v)
    ab.put(cache, 0, [at], 0, np.zeros((1, 1, 128), np.float32))
    rows = Rows(rng, cache, 24, [0] * ROWS)
    assert rows.call(row_ke=torch.full((ROWS,), n, dtype=torch.int32, device=DEV)) == 0
    out = rows.dev["out"].float().cpu().numpy()
    assert np.array_equal(np.isposinf(out), np.broadcast_to(np.isin(np.arange(128), [5, 64]), out.shape))
    assert np.array_equal(np.isneginf(out), np.broadcast_to(np.arange(128) == 77, out.shape))
    finite = [i for i in range(128) if i not in (5, 64, 77)]
    k, v = cache.tokens(0, np.arange(n))
    want, mean, lse, size = ab.attend(rows.q[0].to(torch.float64).numpy(), k, np.where(np.isinf(v), 0, v), rows.scale)
    off, lse_off = ab.bound(want, mean, size, 128, n)
    assert (np.abs(out[0] - want) <= off)[:, finite].all()
    assert (np.abs(rows.dev["lse"][0].cpu().numpy() - lse) <= lse_off + 2.0 ** -22 * np.abs(lse)).all()


@pytest.mark.parametrize("first", [1, 128, 300])
@pytest.mark.parametrize("heads", [3, 40])
def test_scores_of_minus_infinity_before_others(first, heads):
    """Tokens whose score is minus infinity for half of the heads have no weight there, also where a row begins with
    whole tiles of them and what follows has scores far below zero."""
    rng = np.random.Generator(np.random.PCG64(44))
    n = 600
    cache = ref.Cache(rng, 1, 128, 64, "bf16", [n])
    k = rng.standard_normal((n, 1, 128)).astype(np.float32)
    k[:, 0, 0] = 0
    k[:first, 0, 0] = -np.inf
    k[first:, 0, 1] = -300 * np.sqrt(128)
    ab.put(cache, 0, np.arange(n), 0, k)
    rows = Rows(rng, cache, heads, [0] * ROWS)
    q = rows.q.clone()
    q[:, :, 1] = 1
    q[:, ::2, 0] = 1           # these heads: minus infinity first
    q[:, 1::2, 0] = -1         # these: plus infinity, so NaN
    _queries(rows, q)
    assert rows.call(row_ke=torch.full((ROWS,), n, dtype=torch.int32, device=DEV)) == 0
    out, lse = rows.dev["out"], rows.dev["lse"]
    assert bool(torch.isnan(out[:, 1::2]).all())
    keep = list(range(0, heads, 2))
    kk, vv = cache.tokens(0, np.arange(first, n))
    for r in (0, 77, ROWS - 1):
        ab.check(out[r, keep], lse[r, keep], q[r, keep].to(torch.float64).numpy(), kk, vv, rows.scale)


def test_scores_of_minus_infinity_alone():
    """A head without a score above minus infinity has the result of a row without tokens."""
    rng = np.random.Generator(np.random.PCG64(45))
    cache = ref.Cache(rng, 1, 64, 64, "bf16", [400])
    k = rng.standard_normal((400, 1, 64)).astype(np.float32)
    k[:, 0, 0] = -np.inf
    ab.put(cache, 0, np.arange(400), 0, k)
    rows = Rows(rng, cache, 4, [0] * ROWS)
    q = rows.q.clone()
    q[:, :, 0] = 2
    _queries(rows, q)
    assert rows.call(row_ke=torch.full((ROWS,), 400, dtype=torch.int32, device=DEV)) == 0
    assert bool((rows.dev["out"] == 0).all()) and bool(torch.isneginf(rows.dev["lse"]).all())


@pytest.mark.parametrize("dim", [64, 128])
def test_every_code_of_an_8_bit_cache(dim):
    """Rows of one token, whose result is its values and whose lse is its score: all 256 codes as values, and as keys
    under queries of one element each. NaN codes stay NaN and touch nothing else."""
    rng = np.random.Generator(np.random.PCG64(46))
    seqs = 256 // dim
    cache = ref.Cache(rng, 1, dim, 16, "e4m3", [1] * seqs)
    codes = np.arange(256, dtype=np.uint8).reshape(seqs, 1, 1, dim)
    for s in range(seqs):
        for side in (0, 1):
            ab.put(cache, s, [0], side, codes[s], np.full((1, 1), 0.375, np.float32))
    rows = Rows(rng, cache, dim, list(range(seqs)), scale=0.5)
    values = ref.e4m3_values(codes.reshape(seqs, dim)) * 0.375
    # values: zero queries, so that every key's finite codes give a score of zero; NaN keys make every head NaN
    _queries(rows, torch.zeros(seqs, dim, dim, dtype=torch.bfloat16))
    assert rows.call(row_ke=torch.ones(seqs, dtype=torch.int32, device=DEV)) == 0
    finite = [s for s in range(seqs) if np.isfinite(values[s]).all()]
    for s in finite:
        want = torch.from_numpy(values[s]).to(torch.bfloat16).expand(dim, dim)
        assert torch.equal(rows.dev["out"][s].cpu(), want)
        assert bool((rows.dev["lse"][s] == 0).all())
    for s in set(range(seqs)) - set(finite):
        assert bool(torch.isnan(rows.dev["out"][s]).all())
    # the same with keys of zero: a NaN value is NaN in its element only
    for s in range(seqs):
        ab.put(cache, s, [0], 0, np.zeros((1, 1, dim), np.uint8), np.ones((1, 1), np.float32))
    rows.dev.update(cache.to(DEV))
    assert rows.call(row_ke=torch.ones(seqs, dtype=torch.int32, device=DEV)) == 0
    for s in range(seqs):
        want = torch.from_numpy(values[s]).to(torch.bfloat16).expand(dim, dim)
        got = rows.dev["out"][s].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())
    # keys: head h asks for element h alone
    for s in range(seqs):
        ab.put(cache, s, [0], 0, np.where(np.isnan(values[s]), 0, codes[s]).astype(np.uint8), np.full((1, 1), 0.375, np.float32))
    rows.dev.update(cache.to(DEV))
    _queries(rows, torch.eye(dim, dtype=torch.bfloat16).expand(seqs, dim, dim).contiguous())
    assert rows.call(row_ke=torch.ones(seqs, dtype=torch.int32, device=DEV)) == 0
    want = np.where(np.isnan(values), 0, values) * 0.5
    assert (np.abs(rows.dev["lse"].cpu().numpy() - want) <= 2.0 ** -21 * np.abs(want)).all()
