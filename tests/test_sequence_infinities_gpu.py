"""Values that are not finite under masks: they reach the rows that see them, element by element, and nobody else, and what that
costs does not grow with the context."""

import time

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_bounds as bounds
import sequence_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def _put(b, seq, t, value, rng):
    """An element of a token's value in a bf16 cache, or its scale or its codes in an 8-bit one, of one kv head."""
    c = b.cache
    page, off, g = int(c.table[seq, t // c.page]), t % c.page, int(rng.integers(0, c.kv_heads))
    if c.dtype == "bf16":
        d = int(rng.integers(0, c.dim))
        c.data[page, 1, g, off, d] = value
        c.values[page, 1, g, off, d] = value
    elif np.isnan(value):
        d = int(rng.integers(0, c.dim))
        c.data[page, 1, g, off, d] = 0x7F
        c.values[page, 1, g, off, d] = value
    else:  # (scales are positive)
        c.scales[page, 1, g, off] = np.inf
        with np.errstate(invalid="ignore"):
            c.values[page, 1, g, off] = np.sign(c.values[page, 1, g, off]) * np.inf  # a code of zero: NaN


def _too_small(q, k, v, scale):
    """Elements [H, D] of a row that meet a value that is not finite with a weight below fp32's smallest normal number: the
    library says NaN there, or infinite."""
    h, d = q.shape
    s = np.einsum("gid,tgd->git", q.reshape(k.shape[1], -1, d), k) * scale
    tiny = (s - s.max(-1, keepdims=True)) * np.log2(np.e) < -125
    return np.einsum("git,tgd->gid", tiny.astype(int), (~np.isfinite(v)).astype(int)).reshape(h, d) > 0


def _check(b, sets):
    """Every element: finite and within the bound where the formula is, infinite or NaN where it is."""
    q, out, lse = (x.to(torch.float64).cpu().numpy() for x in (b.q, b.out, b.lse))
    odd = 0
    for s, per in enumerate(sets):
        for i, at in enumerate(per):
            r = int(b.cu[s]) + i
            if len(at) == 0:
                assert (out[r] == 0).all()
                continue
            k, v = b.cache.tokens(s, at)
            with np.errstate(invalid="ignore"):
                want, mean, want_lse, size = ref.attend(q[r], k, v, b.scale)
                fine = np.isfinite(want)
                off, lse_off = ref.bound(np.where(fine, want, 0), np.where(fine, mean, 0), size, b.dim, len(at))
                same = (out[r] == want) | (np.isnan(out[r]) & (np.isnan(want) | _too_small(q[r], k, v, b.scale)))
                assert same[~fine].all(), (s, i)
            odd += (~fine).any()
            assert np.isfinite(out[r][fine]).all(), (s, i)
            assert (np.abs(out[r][fine] - want[fine]) <= off[fine]).all(), (s, i)
            assert (np.abs(lse[r] - want_lse) <= lse_off + 2.0 ** -22 * np.abs(want_lse)).all(), (s, i)
    assert odd > 0


GEOMETRIES = [  # heads, kv heads, dim, page, dtype
    (64, 8, 128, 64, "bf16"), (4, 4, 128, 16, "bf16"), (24, 1, 64, 32, "bf16"), (128, 1, 128, 64, "bf16"), (33, 1, 64, 5, "bf16"),
    (64, 8, 128, 64, "e4m3"), (6, 2, 64, 16, "e4m3"), (41, 1, 128, 24, "e4m3"),
]
# one tile of queries and two; all tiles masked, the first or the last one; contexts that several CTAs share
SEQS = [(3, 300), (1, 200), (40, 1000), (130, 400), (7, 7), (2, 129), (70, 70), (4, 2500), (300, 300)]


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
@pytest.mark.parametrize("window,sinks", [(150, 3), (2 ** 31 - 1, 0), (20, 140)])
def test_windows(heads, kv_heads, dim, page, dtype, window, sinks):
    rng = _rng(heads, dim, window, sinks)
    b = ref.Batch(rng, heads, kv_heads, dim, page, dtype, SEQS)
    sets = [ref.window_sets(n, length, window, sinks) for n, length in SEQS]
    for s, (n, length) in enumerate(SEQS):
        near = [length - 1 - int(rng.integers(0, min(length, n + 5))) for _ in range(3)]  # the newest tokens, seen by the last rows
        low = [max(0, min(length - 1, length - n - window + int(rng.integers(0, n + 3)))), min(2, length - 1)]
        for j, t in enumerate(near + low):
            if rng.random() < 0.6:
                _put(b, s, t, (np.inf, -np.inf, np.nan, np.inf, np.nan)[j], rng)
    assert b.call(window=window, sinks=sinks) == 0
    _check(b, sets)


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
def test_trees(heads, kv_heads, dim, page, dtype):
    rng = _rng(heads, dim, 5)
    b = ref.Batch(rng, heads, kv_heads, dim, page, dtype, SEQS)
    masks = []
    for s, (n, length) in enumerate(SEQS):
        masks += [{j for j in range(n) if rng.random() < 0.5} for _ in range(n)] if s % 2 else ref.random_tree(rng, n)
        for value in (np.inf, np.nan, -np.inf):
            _put(b, s, length - 1 - int(rng.integers(0, n)), value, rng)
        if s % 3 == 0:
            _put(b, s, int(rng.integers(0, length)), np.inf, rng)  # of the context, for most
    words = -(-max(n for n, _ in SEQS) // 32)
    assert b.call(tree_mask=ref.pack(masks + [set()] * 2, words)) == 0
    _check(b, [ref.tree_sets(n, length, masks[b.cu[s]:b.cu[s] + n]) for s, (n, length) in enumerate(SEQS)])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_long_context_does_not_pay(dtype):
    """Sixteen trees of 64 nodes behind 30000 tokens, NaN in a drafted value of each and an infinite value early in each
    context, which all rows see. An item is a sequence's 32 rows on one of 8 kv heads, so there are 256 on 152 SMs or more, cut
    into two or three each. The values that some rows do not see lie in an item's last one or two tiles, and a tile by hand is
    8 * 128 rounds of some 45 instructions for each of 8 warps on 4 schedulers: 50 us at one instruction a cycle, 500 us at
    a tenth of that. Two tiles of three items are 3 ms, and 20 for a call leave room for a slow clock. Summed over the whole
    context, as 240 tiles, it would be a hundred times that."""
    rng = _rng(8)
    n, length, seqs = 64, 30000, 16
    plan = smq.AttentionPlan(64, 8, 128, 64, max_rows=n * seqs, cache_dtype=dtype)
    columns = -(-length // 64)
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(seqs * columns, 2, 8, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
    scales = None
    if dtype == "e4m3":
        x = x.to(torch.float8_e4m3fn).view(torch.uint8)
        scales = torch.ones(seqs * columns, 2, 8, 64, device=DEV)
    table = torch.arange(seqs * columns, dtype=torch.int32, device=DEV).view(seqs, columns)
    masks = [m for _ in range(seqs) for m in ref.random_tree(rng, n)]
    mask = torch.from_numpy(ref.pack(masks, 2)).to(DEV)
    q = torch.randn(n * seqs, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(n * seqs, 64, device=DEV)
    ws = plan.sequence_workspace()
    cu = torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * n
    lens = torch.full((seqs,), length, dtype=torch.int32, device=DEV)
    call = smq.SequenceAttentionCall(plan, q, x[:, 0], x[:, 1], table, cu, lens, n, out, ws, tree_mask=mask, lse=lse,
                                     k_scales=None if scales is None else scales[:, 0],
                                     v_scales=None if scales is None else scales[:, 1])
    call()
    clean, clean_lse = out.clone(), lse.clone()
    early = 5
    for s in range(seqs):
        node = length - n + 1 + s % 40
        page = int(table[s, node // 64])
        first = int(table[s, early // 64])
        if dtype == "bf16":
            x[page, 1, :, node % 64, 9] = float("nan")
            x[first, 1, :, early % 64, 100] = float("inf")
        else:
            x[page, 1, :, node % 64, 9] = 0x7F
            x[first, 1, :, early % 64, 100] = 0x7F
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert smq.smq_get_status(ws) == 0
    assert torch.equal(lse, clean_lse), "the weights are the same"
    sees = torch.tensor([1 + r // n % 40 in masks[r] for r in range(n * seqs)], device=DEV)
    assert 0 < int(sees.sum()) < len(sees)
    assert torch.isnan(out[sees][:, :, 9]).all() and torch.isfinite(out[~sees][:, :, 9]).all()
    assert not torch.isfinite(out[:, :, 100]).any()
    rest = [d for d in range(128) if d not in (9, 100)]
    # the tile by hand adds the same products in another order: a step of bf16, of results below 4
    assert (out[:, :, rest].float() - clean[:, :, rest].float()).abs().max() <= 2.0 ** -6
    assert (out[~sees][:, :, 9].float() - clean[~sees][:, :, 9].float()).abs().max() <= 2.0 ** -6
    assert took < 0.02, took


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [2, 64])
def test_with_scores_far_from_zero(dtype, heads):
    """Both rare ways of a tile at once: scores past 1e12, of which the largest share all the weight, and values that some rows do not
    see. A row's weights are those of equal scores, so roundings of scores do not matter."""
    rng = _rng(heads, 3)
    seqs = [(20, 250), (3, 100), (45, 300)]
    b = ref.Batch(rng, heads, 1, 128, 64, dtype, seqs, scale=1.0)
    b.q[:] = 0
    b.q[:, :, 3] = torch.from_numpy(rng.choice([-3e12, 3e12, 0.5], b.q.shape[:2])).to(torch.bfloat16)
    masks = []
    for i, (n, length) in enumerate(seqs):
        keys = np.zeros((length, 1, 128))
        keys[:, :, 3] = rng.integers(1, 4, (length, 1))
        bounds.put(b.cache, i, np.arange(length), 0, keys)
        masks += ref.random_tree(rng, n)
        for value in (np.nan, np.inf):
            t = length - 1 - int(rng.integers(0, n - 1))
            page, off = b.cache.table[i][t // 64], t % 64
            if dtype == "bf16":
                b.cache.data[page, 1, 0, off, 7] = value
            else:
                b.cache.data[page, 1, 0, off, 7] = 0x7F
            b.cache.values[page, 1, 0, off, 7] = value if dtype == "bf16" else np.nan
    assert b.call(tree_mask=ref.pack(masks + [set()] * 2, 2)) == 0
    out = b.out.double().cpu().numpy()
    sets = [ref.tree_sets(n, length, masks[b.cu[i]:b.cu[i] + n]) for i, (n, length) in enumerate(seqs)]
    clean = 0
    for i, per in enumerate(sets):
        for r, at in zip(range(b.cu[i], b.cu[i + 1]), per):
            k, v = b.cache.tokens(i, at)
            odd = ~np.isfinite(v[:, 0]).all(0)  # by element
            v = np.where(np.isfinite(v), v, 0)
            want, mean, _, _ = ref.attend(b.q[r].double().numpy(), k, v, 1.0)
            off, _ = ref.bound(want, mean, np.zeros(heads), 128, len(at))
            assert (np.abs(out[r] - want) <= off)[:, ~odd].all(), (i, r)
            assert not np.isfinite(out[r][:, odd]).any(), (i, r)
            clean += not odd.any()
    assert 0 < clean < len(masks)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("tile", [0, 1])  # of the first CTA, which has two: 5 * 2 * 8 items of 3 or 4 tiles over 152
def test_a_withheld_tile_beside_such_values(dtype, tile):
    rng = _rng(tile)
    seqs = [(40, 700)] * 5
    b = ref.Batch(rng, 64, 8, 128, 64, dtype, seqs)
    sets = [ref.window_sets(n, length, 300, 4) for n, length in seqs]
    for s in range(5):
        for t in (5, 375, 520, 690):
            _put(b, s, t, np.nan, rng)
    b.plan.set_wait_limit(2_000_000)
    b.plan.inject_stall(tile)
    assert b.call(window=300, sinks=4) & smq.SMQ_ERR_TIMEOUT
    b.plan.inject_stall(-1)
    b.plan.set_wait_limit(2_000_000_000)
    assert b.call(window=300, sinks=4) == 0
    _check(b, sets)
