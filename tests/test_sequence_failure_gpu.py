"""The sequences' attention when a wait runs out, without a fault: a withheld hand-off, and a limit that any call overruns. Then
long runs of tiles, calls at once, and the whole loop of a drafting step."""

import time

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import sequence_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


@pytest.mark.parametrize("heads,kv_heads,dtype,seqs,tile", [
    (64, 8, "bf16", [(1, 700)] * 20, 0), (64, 8, "bf16", [(40, 700)] * 5, 2), (64, 8, "e4m3", [(2, 900)] * 20, 1),
    (32, 1, "e4m3", [(30, 2000)] * 9, 1), (16, 16, "bf16", [(1, 3000)] * 40, 5),
])
def test_a_withheld_tile_times_out_and_the_next_call_is_right(heads, kv_heads, dtype, seqs, tile):
    b = ref.Batch(_rng(heads, tile), heads, kv_heads, 128, 64, dtype, seqs)
    sets = [ref.window_sets(n, length, 600, 4) for n, length in seqs]
    b.plan.set_wait_limit(2_000_000)
    b.plan.inject_stall(tile)
    t0 = time.perf_counter()
    assert b.call(window=600, sinks=4) & smq.SMQ_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    b.plan.inject_stall(-1)
    b.plan.set_wait_limit(2_000_000_000)
    assert b.call(window=600, sinks=4) == 0
    b.check(sets)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 60])
def test_a_limit_that_any_call_overruns(dtype, rows):
    """Waits of a nanosecond: calls end all the same, and leave nothing behind for the next one."""
    seqs = [(rows, 2000 + 60 * i) for i in range(6)]
    b = ref.Batch(_rng(rows), 64, 8, 128, 64, dtype, seqs)
    sets = [ref.window_sets(n, length, 1500, 4) for n, length in seqs]
    for _ in range(5):
        b.plan.set_wait_limit(1)
        b.call(window=1500, sinks=4)  # times out, or not: some waits find their phase complete
        b.plan.set_wait_limit(2_000_000_000)
        assert b.call(window=1500, sinks=4) == 0
    b.check(sets, rows={0, rows - 1})


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype,n", [
    (64, 8, 128, 64, "e4m3", 2), (64, 8, 128, 64, "bf16", 2), (32, 1, 64, 32, "e4m3", 30), (8, 8, 64, 16, "bf16", 1),
    (64, 1, 128, 64, "e4m3", 9),
])
def test_many_tiles_for_each_cta(heads, kv_heads, dim, page, dtype, n):
    """Every place of the rings in use many times over, segments of every length among them."""
    rng = _rng(heads, n, dim)
    seqs = [(n, 6000 - 7 * i) for i in range(24)] + [(n, n), (1, 1), (n, 300)]
    b = ref.Batch(rng, heads, kv_heads, dim, page, dtype, seqs)
    b.tree([m for r, _ in seqs for m in ref.random_tree(rng, r)])


@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [(64, 8, 64, "bf16"), (4, 4, 64, "bf16"), (64, 8, 128, "bf16"),
                                                      (16, 8, 64, "e4m3"), (64, 8, 128, "e4m3")])
@pytest.mark.parametrize("rows", [1, 3])
def test_many_items_of_one_tile(heads, kv_heads, dim, dtype, rows):
    """Short contexts, one tile each, so that tile after tile is the same stream's; sixty calls with the same bits."""
    rng = _rng(heads, dim, rows)
    seqs = [(rows, rows + int(rng.integers(0, 120))) for _ in range(700)]
    b = ref.Batch(rng, heads, kv_heads, dim, 32, dtype, seqs)
    b.window(1000)
    first = b.out.clone(), b.lse.clone()
    for _ in range(60):
        b.out.fill_(3)
        b.made()
        assert torch.equal(first[0][:-2], b.out[:-2]) and torch.equal(first[1], b.lse)
    assert smq.smq_get_status(b.workspace) == 0


def test_two_calls_at_once():
    """Two streams, a workspace each, over one cache; sixteen rounds, the same bits every time."""
    rng = _rng(5)
    seqs = [(30, 5000), (1, 3000), (64, 700)]
    b = ref.Batch(rng, 64, 8, 128, 64, "bf16", seqs)
    sets = b.window(2000, 4, poison=False)
    want = b.out.clone(), b.lse.clone()
    args = dict(b.cache.to(DEV), block_table=torch.from_numpy(b.table).to(DEV), cu_rows=torch.from_numpy(b.cu).to(DEV),
                seq_indices=torch.from_numpy(b.order).to(DEV), max_seq_rows=64, window=2000, sinks=4,
                seq_len=torch.tensor([x for _, x in seqs], dtype=torch.int32, device=DEV))
    outs = [(torch.full_like(b.out, 9), torch.full_like(b.lse, 9)) for _ in range(2)]
    calls = [smq.SequenceAttentionCall(b.plan, b.q_dev, out=o, lse=x, workspace=b.plan.sequence_workspace(), **args) for o, x in outs]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(16):
        for s, call in zip(streams, calls):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    for o, x in outs:
        assert torch.equal(o, want[0]) and torch.equal(x, want[1])
    assert sets


def test_a_drafting_step_from_pages_to_compaction():
    """resize, append, tree attention, compact, resize: the accepted path is what plain decoding of it would have left."""
    rng = _rng(6)
    heads, kv_heads, dim, page, rows, nodes = 16, 2, 64, 16, 5, 9
    pages, columns = 120, 20
    pool = smq.PagePlan(page, pages, rows, columns)
    refs, table = pool.state()
    pool_ws = pool.workspace()
    plan = smq.AttentionPlan(heads, kv_heads, dim, page, max_rows=256)
    ws, seq_ws = plan.workspace(), plan.sequence_workspace()
    data = torch.full((pages, 2, kv_heads, page, dim), float("nan"), device=DEV, dtype=torch.bfloat16)
    sides = dict(k_cache=data[:, 0], v_cache=data[:, 1])
    lens = np.array([0, 16, 33, 100, 200])

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)

    def slots(row, at):
        t = table.cpu().numpy()
        return torch.tensor([int(t[r, p // page]) * page + int(p % page) for r, p in zip(row, at)], device=DEV)

    def append(row, at, k, v):
        smq.sparse_mqa_append_kv(plan, None, k, v, None, None, slots(row, at), workspace=ws, **sides)

    def some(n):
        return ref.bounds.bf16(rng.standard_normal((n, kv_heads, dim)))

    keys, values = [some(n) for n in lens], [some(n) for n in lens]
    smq.sparse_mqa_pages_resize(pool, refs, table, i32(lens + nodes), pool_ws)
    for r, n in enumerate(lens):
        if n:
            append([r] * n, range(n), keys[r].to(DEV), values[r].to(DEV))
    draft_k, draft_v = [some(nodes) for _ in lens], [some(nodes) for _ in lens]
    trees = [ref.random_tree(rng, nodes) for _ in lens]
    for r, n in enumerate(lens):
        append([r] * nodes, range(n, n + nodes), draft_k[r].to(DEV), draft_v[r].to(DEV))
    q = ref.bounds.bf16(rng.standard_normal((rows * nodes, heads, dim)))
    out, lse = torch.empty(rows * nodes, heads, dim, device=DEV, dtype=torch.bfloat16), torch.empty(rows * nodes, heads, device=DEV)
    cu = i32(np.arange(rows + 1) * nodes)
    smq.sparse_mqa_attention_tree(plan, q.to(DEV), block_table=table, cu_rows=cu, seq_len=i32(lens + nodes), max_seq_rows=nodes,
                                  out=out, workspace=seq_ws, tree_mask=i32(ref.pack([m for t in trees for m in t], 1)), lse=lse, **sides)
    # accept the path to the last node, and check its rows
    paths = [sorted(t[-1]) for t in trees]
    for r, path in enumerate(paths):
        for node in path:
            at = sorted(trees[r][node])
            k = torch.cat([keys[r], draft_k[r][at]]).double().numpy()
            v = torch.cat([values[r], draft_v[r][at]]).double().numpy()
            want, mean, want_lse, size = ref.attend(q[r * nodes + node].double().numpy(), k, v, dim ** -0.5)
            off, _ = ref.bound(want, mean, size, dim, len(k))
            assert (np.abs(out[r * nodes + node].double().cpu().numpy() - want) <= off).all(), (r, node)
    keep = np.full((rows, nodes), -1)
    for r, path in enumerate(paths):
        keep[r, :len(path)] = lens[r] + np.array(path)
    smq.sparse_mqa_cache_compact(pool, refs, table, i32(lens), i32(keep), [data[:, 0], data[:, 1]], pool_ws)
    after = lens + np.array([len(x) for x in paths])
    smq.sparse_mqa_pages_resize(pool, refs, table, i32(after), pool_ws)
    assert smq.smq_get_status(ws) == smq.smq_get_status(seq_ws) == smq.smq_get_status(pool_ws) == 0
    t = table.cpu().numpy()
    assert int(refs.sum()) == (t >= 0).sum() == sum(-(-n // page) for n in after)
    for r, path in enumerate(paths):
        at = np.arange(after[r])
        where, off = torch.tensor(t[r][at // page]).long(), torch.tensor(at % page)
        for side, parts in ((0, (keys[r], draft_k[r][path])), (1, (values[r], draft_v[r][path]))):
            got = data.cpu()[where, side, :, off]
            assert torch.equal(got.view(torch.int16), torch.cat(parts).view(torch.int16)), (r, side)
    # the next token of every sequence sees the compacted context: a window call and the plain decode call agree
    q1 = ref.bounds.bf16(rng.standard_normal((rows, heads, dim))).to(DEV)
    one, whole = torch.empty_like(q1), torch.empty_like(q1)
    smq.sparse_mqa_attention_window(plan, q1, block_table=table, cu_rows=i32(np.arange(rows + 1)), seq_len=i32(after), max_seq_rows=1,
                                    out=one, workspace=seq_ws, window=1000, **sides)
    smq.sparse_mqa_attention_decode(plan, q1, block_table=table, row_indices=None, row_ke=i32(after), out=whole, workspace=ws, **sides)
    # weights of 8 bits against 16, means of |v| below 4: 2^-8 of each, and the results' own rounding
    assert (one.float() - whole.float()).abs().max() <= 2 ** -8 * 4 + 2 ** -7 * whole.float().abs().max()
