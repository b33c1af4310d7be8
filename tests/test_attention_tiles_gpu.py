"""Long runs of tiles within a CTA: running maxima that move many times, rings and buffers that wrap, and ordinary rows,
all within the bound of the kernel's own arithmetic."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_bounds as ab
import attention_ref as ref
from test_attention_gpu import GEOMETRIES, Rows

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _check(rows, r, positions):
    k, v = rows.cache.tokens(rows.seqs[r], positions)
    ab.check(rows.dev["out"][r], rows.dev["lse"][r], rows.q[r].to(torch.float64).numpy(), k, v, rows.scale, f"row {r}")


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("course", ["rise", "fall", "waves"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [16, 17, 40, 64, 100, 128])
def test_a_maximum_that_moves_within_a_row(heads, dim, dtype, course):
    """Two rows and more of 12 tiles a CTA, over one sequence whose keys lean towards one direction: more and more, less
    and less, or back and forth. The queries follow it with strengths of both signs."""
    n = 1500
    rng = np.random.Generator(np.random.PCG64(heads + dim))
    cache = ref.Cache(rng, 1, dim, 64, dtype, [n])
    lean = np.linspace(0, 1, n)
    lean = {"rise": lean, "fall": 1 - lean, "waves": np.sin(lean * 20)}[course]
    k = (rng.standard_normal((n, 1, dim)) * 0.3).astype(np.float32)
    k[:, 0, 5] += 12 * lean
    ab.put(cache, 0, np.arange(n), 0, k)
    count = 2 * _sms() + 3
    rows = Rows(rng, cache, heads, [0] * count)
    q = rows.q.clone()
    q[:, :, 5] = torch.linspace(-60, 60, heads).to(torch.bfloat16)
    rows.q, rows.q_dev = q, q.to(DEV)
    assert rows.call(row_ke=_i32([n] * count)) == 0
    for r in (0, 1, 2, count // 2, count - 1):
        _check(rows, r, np.arange(n))


@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [
    (16, 1, 128, "e4m3"), (40, 1, 64, "e4m3"), (64, 1, 128, "e4m3"), (128, 1, 128, "e4m3"), (100, 1, 64, "e4m3"),
    (24, 3, 128, "e4m3"), (64, 1, 128, "bf16"), (128, 1, 64, "bf16"),
])
def test_many_short_rows_of_a_cta(heads, kv_heads, dim, dtype):
    """More than 20 rows of one or two tiles a CTA, so that every ring and buffer of segments, tiles and queries wraps."""
    rng = np.random.Generator(np.random.PCG64(heads))
    lens = [1, 100, 128, 129, 250, 17, 0, 64]
    cache = ref.Cache(rng, kv_heads, dim, 32, dtype, lens)
    count = 24 * _sms() // kv_heads + 5
    seqs = [int(s) for s in rng.integers(0, len(lens), count)]
    rows = Rows(rng, cache, heads, seqs)
    assert rows.call(row_ke=_i32([lens[s] for s in seqs])) == 0
    for r in list(range(0, count, count // 40)) + [count - 1]:
        if lens[seqs[r]]:
            _check(rows, r, np.arange(lens[seqs[r]]))
        else:
            assert bool((rows.dev["out"][r] == 0).all()) and bool(torch.isneginf(rows.dev["lse"][r]).all())
    ids = np.stack([rng.integers(-1, max(lens[s], 1), 30) if lens[s] else np.full(30, -1) for s in seqs]).astype(np.int32)
    assert rows.call(token_ids=torch.from_numpy(ids).to(DEV)) == 0
    for r in range(0, count, count // 40):
        if (ids[r] >= 0).any():
            _check(rows, r, ids[r][ids[r] >= 0])


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
def test_ordinary_rows_within_the_bound(heads, kv_heads, dim, page, dtype):
    rng = np.random.Generator(np.random.PCG64(heads + 5 * dim))
    lens = [1, 2, 127, 128, 129, 300, 1000]
    cache = ref.Cache(rng, kv_heads, dim, page, dtype, lens)
    rows = Rows(rng, cache, heads, list(range(len(lens))))
    assert rows.call(row_ke=_i32(lens)) == 0
    for r, n in enumerate(lens):
        _check(rows, r, np.arange(n))
    ids = np.stack([rng.integers(0, n, 400) for n in lens]).astype(np.int32)
    assert rows.call(token_ids=torch.from_numpy(ids).to(DEV)) == 0
    for r in range(len(lens)):
        _check(rows, r, ids[r])
