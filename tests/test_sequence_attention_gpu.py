"""Attention of sequences' query rows, through the public entry points, against plain 64-bit forms: a sliding window with
sinks, and trees of drafted tokens. What a row does not see is poisoned, or its page is not there."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_bounds as bounds
import sequence_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"

GEOMETRIES = [  # heads, kv heads, dim, page, dtype
    (64, 8, 128, 64, "bf16"), (1, 1, 128, 64, "bf16"), (16, 16, 64, 16, "bf16"), (24, 1, 64, 32, "bf16"), (33, 1, 128, 5, "bf16"),
    (128, 1, 128, 128, "bf16"), (130, 2, 64, 64, "bf16"), (6, 2, 128, 1, "bf16"),
    (64, 8, 128, 64, "e4m3"), (2, 1, 64, 64, "e4m3"), (41, 1, 64, 24, "e4m3"), (128, 1, 128, 32, "e4m3"), (12, 4, 128, 7, "e4m3"),
]

# rows and length: one and many, prefills from the start, no rows, no context, a negative start
SEQS = [(1, 1), (3, 300), (0, 50), (7, 7), (1, 700), (40, 131), (0, 0), (5, 3), (2, 0), (67, 67), (1, 128), (9, 129)]


def _rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 0)])
def test_window_matches(heads, kv_heads, dim, page, dtype, window, sinks):
    ref.Batch(_rng(heads, dim, window), heads, kv_heads, dim, page, dtype, SEQS).window(window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 1), (2, 130), (127, 0), (128, 3), (129, 128), (64, 700), (2 ** 31 - 1, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (300, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_windows_and_sinks_of_every_size(window, sinks, dtype):
    ref.Batch(_rng(window, sinks), 8, 2, 64, 16, dtype, SEQS + [(130, 500), (20, 1000)]).window(window, sinks)


@pytest.mark.parametrize("heads,kv_heads,dtype,seqs,window,sinks", [
    (8, 1, "bf16", [(1, 30011)], 30000, 0),               # one row over every CTA
    (64, 8, "bf16", [(600, 700)], 256, 4),                # a prefill chunk
    (16, 1, "e4m3", [(300, 2000), (1, 9000), (33, 40)], 5000, 64),
    (1, 1, "bf16", [(1000, 1000)], 700, 2),               # 256 rows a block, the first ones of a context
    (128, 1, "bf16", [(21, 1500)], 1024, 16),
    (3, 1, "bf16", [(500, 900), (1, 1)], 130, 129),
])
def test_window_of_long_sequences(heads, kv_heads, dtype, seqs, window, sinks):
    b = ref.Batch(_rng(heads, window), heads, kv_heads, 128, 64, dtype, seqs)
    b.window(window, sinks)
    first = b.out.clone(), b.lse.clone()
    b.made()
    assert torch.equal(first[0], b.out) and torch.equal(first[1], b.lse), "the same bits again"


def test_many_sequences():
    rng = _rng(12)
    seqs = [(int(rng.integers(0, 4)), int(rng.integers(0, 300))) for _ in range(1400)]
    ref.Batch(rng, 4, 2, 64, 16, "bf16", seqs).window(50, 3)


@pytest.mark.parametrize("heads,kv_heads,dtype", [(64, 8, "bf16"), (12, 2, "e4m3"), (128, 1, "bf16")])
def test_many_sequences_of_many_blocks(heads, kv_heads, dtype):
    """More sequences than a warp's lanes, of none to several blocks of rows each."""
    rng = _rng(13, heads)
    seqs = []
    for i in range(150):
        n = int(rng.integers(0, 70)) if i % 3 else int(rng.integers(0, 2))
        seqs.append((n, n + int(rng.integers(0, 200))))
    ref.Batch(rng, heads, kv_heads, 64, 16, dtype, seqs).window(90, 5)


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
def test_tree_matches(heads, kv_heads, dim, page, dtype):
    rng = _rng(heads, dim, 9)
    b = ref.Batch(rng, heads, kv_heads, dim, page, dtype, SEQS)
    b.tree([m for n, _ in SEQS for m in ref.random_tree(rng, n)])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_masks_of_any_bits(dtype):
    """Rows without a bit, rows with every bit, bits past the sequence's rows, more words than nodes."""
    rng = _rng(4)
    seqs = [(1, 1), (64, 64), (33, 200), (100, 777), (5, 5), (31, 500), (3, 2)]
    masks = []
    for n, _ in seqs:
        for i in range(n):
            masks.append([set(), set(range(160)), {n - 1}, {j for j in range(160) if rng.random() < 0.5}][i % 4])
    ref.Batch(rng, 8, 2, 128, 64, dtype, seqs).tree(masks, words=5)


@pytest.mark.parametrize("heads,kv_heads,dtype,seqs", [
    (64, 8, "bf16", [(64, 9000)]), (64, 1, "e4m3", [(25, 4000), (7, 100)]), (128, 1, "bf16", [(1000, 1100)]),
    (8, 8, "bf16", [(130, 5000), (2, 2)]),
])
def test_tree_of_long_sequences(heads, kv_heads, dtype, seqs):
    rng = _rng(heads)
    b = ref.Batch(rng, heads, kv_heads, 128, 64, dtype, seqs)
    b.tree([m for n, _ in seqs for m in ref.random_tree(rng, n)])
    first = b.out.clone(), b.lse.clone()
    b.made()
    assert torch.equal(first[0], b.out) and torch.equal(first[1], b.lse), "the same bits again"


def test_a_window_of_one_row_is_the_decode_call():
    """A row whose window covers its context has what sparse_mqa_attention_decode has, up to rounding."""
    rng = _rng(3)
    lens = [1, 200, 1000]
    b = ref.Batch(rng, 16, 2, 128, 64, "bf16", [(1, n) for n in lens], pad=0)
    b.window(2000)
    out = torch.empty_like(b.out)
    smq.sparse_mqa_attention_decode(b.plan, b.q_dev, block_table=torch.from_numpy(b.table).to(DEV),
                                    row_indices=torch.from_numpy(b.order).to(DEV),
                                    row_ke=torch.tensor(lens, dtype=torch.int32, device=DEV), out=out, workspace=b.plan.workspace(),
                                    **b.cache.to(DEV))
    # weights of 8 bits against weights of 16, means of |v| below 3, results of a few units: 2^-8 of each
    assert (out.float() - b.out.float()).abs().max() <= 2 ** -8 * 3 + 2 ** -7 * out.float().abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("growth", [1, -1])
@pytest.mark.parametrize("heads", [40, 4])
def test_scores_that_rise_and_fall(dtype, growth, heads):
    """Large scores that grow or shrink along the context: the running maximum moves many times, or never again."""
    rng = _rng(15)
    seqs = [(4, 1500)]
    b = ref.Batch(rng, heads, 1, 128, 64, dtype, seqs)
    lean = np.linspace(0, 1, 1500)[::growth]
    keys = b.cache.values[b.cache.table[0][np.arange(1500) // 64], 0, :, np.arange(1500) % 64] * 0.3
    keys[:, :, 5] += 12 * lean[:, None]
    bounds.put(b.cache, 0, np.arange(1500), 0, keys)
    strength = torch.linspace(-60, 60, 4 * heads).view(4, heads)
    b.q[:4, :, 5] = strength.to(torch.bfloat16)
    b.window(1200, 7)


def test_scores_of_minus_infinity():
    """A head whose scores are all minus infinity has no result, one that has some later starts there."""
    rng = _rng(8)
    b = ref.Batch(rng, 4, 1, 128, 64, "bf16", [(2, 400), (2, 150)])
    b.q[:] = 0
    b.q[:, :, 3] = 1  # every score is key element 3
    for s, n in enumerate((400, 150)):
        keys = rng.standard_normal((n, 1, 128))
        keys[: (300 if s == 0 else 150), :, 3] = -np.inf
        bounds.put(b.cache, s, np.arange(n), 0, keys)
    assert b.call(window=1000) == 0
    sets = ref.window_sets(2, 400, 1000, 0)
    b.check([[s[s >= 300] for s in sets], [np.zeros(0, np.int64)] * 2])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [2, 64])
def test_infinite_values_reach_only_rows_that_see_them(dtype, heads):
    """A drafted token with an infinite value, and one with NaN: their own subtrees and nobody else."""
    rng = _rng(77)
    n, length = 20, 250
    b = ref.Batch(rng, heads, 1, 128, 64, dtype, [(n, length), (n, length)])
    masks = ref.random_tree(rng, n)
    for seq in (0, 1):
        for node, value in ((4, np.inf), (11, np.nan), (17, -np.inf)):
            page, off = b.cache.table[seq][(length - n + node) // 64], (length - n + node) % 64
            if dtype == "bf16":
                b.cache.data[page, 1, 0, off, 7] = float(value)
            else:
                b.cache.scales[page, 1, 0, off] = float(value)  # the whole value is infinite, or NaN
    words = 1
    packed = ref.pack(masks * 2 + [set()] * 2, words)
    assert b.call(tree_mask=packed) == 0
    touched = [i for i, m in enumerate(masks) if m & {4, 11, 17}]
    sets = [ref.tree_sets(n, length, masks)] * 2
    b.check(sets, skip=[s * n + i for s in (0, 1) for i in touched])
    out = b.out.float().cpu()
    assert 0 < len(touched) < n
    for s in (0, 1):
        for i in touched:
            assert not torch.isfinite(out[s * n + i, :, 7]).any()
            if dtype == "bf16":
                rest = torch.cat([out[s * n + i, :, :7], out[s * n + i, :, 8:]], -1)
                assert torch.isfinite(rest).all()
                if masks[i] & {4, 11, 17} == {4}:
                    assert (out[s * n + i, :, 7] == float("inf")).all()


def test_infinite_values_at_the_window_s_edge():
    """Tokens that leave the window one row after the other."""
    rng = _rng(78)
    n, length, window = 40, 500, 128
    b = ref.Batch(rng, 8, 2, 64, 16, "bf16", [(n, length)])
    bad = [length - n - window + 10, length - 15]  # seen by the first ten rows; by the last fifteen
    for t in bad:
        page, off = b.cache.table[0][t // 16], t % 16
        b.cache.data[page, 1, :, off] = float("inf")
    sets = ref.window_sets(n, length, window, 2)
    assert b.call([sets], window=window, sinks=2) == 0
    skip = [i for i, s in enumerate(sets) if set(bad) & set(s.tolist())]
    assert 0 < len(skip) < n
    b.check([sets], skip=skip)
    assert torch.isinf(b.out[skip].float()).all()


def test_masked_keys_do_not_matter():
    rng = _rng(79)
    n, length = 9, 140
    b = ref.Batch(rng, 8, 1, 128, 64, "bf16", [(n, length)])
    masks = ref.random_tree(rng, n)
    for t, value in ((length - n + 5, float("nan")), (length - n + 7, float("inf"))):
        b.cache.data[b.cache.table[0][t // 64], 0, 0, t % 64] = value
    assert b.call(tree_mask=ref.pack(masks + [set()] * 2, 1)) == 0
    b.check([ref.tree_sets(n, length, masks)], skip=[i for i, m in enumerate(masks) if m & {5, 7}])


def test_softmax_scale_and_identity_table():
    b = ref.Batch(_rng(8), 8, 2, 64, 64, "bf16", [(3, 150), (1, 33), (20, 260)], scale=-0.31)
    b.window(140, 5)


def test_bad_sequences_and_pages():
    """A sequence that is refused leaves its rows, the others have theirs; a page that is not there is left out."""
    rng = _rng(30)
    seqs = [(3, 200), (8, 200), (2, 300), (4, 100)]
    b = ref.Batch(rng, 8, 1, 128, 64, "bf16", seqs)
    sets = [ref.window_sets(n, length, 150, 4) for n, length in seqs]
    assert b.call(window=150, sinks=4, max_seq_rows=5) == smq.SMQ_ERR_BOUNDS  # sequence 1 has more
    assert (b.out[3:11] == 9).all() and (b.lse[3:11] == 9).all()
    b.check([sets[0], [], sets[2], sets[3]])
    for page in (-1, -7, b.cache.pages, 2 ** 31 - 1):
        c = ref.Batch(_rng(31), 8, 1, 128, 64, "bf16", seqs)
        c.table[c.order[2], 3] = page  # positions 192 to 255
        assert c.call(window=150, sinks=4) == smq.SMQ_ERR_BOUNDS
        keep = list(sets)
        keep[2] = [s[(s < 192) | (s >= 256)] for s in sets[2]]
        c.check(keep)
    c = ref.Batch(_rng(32), 8, 1, 128, 64, "bf16", seqs)
    c.order[0] = 4  # no such table row
    assert c.call(window=150, sinks=4) == smq.SMQ_ERR_BOUNDS
    none = np.zeros(0, np.int64)
    c.check([[none] * 3] + sets[1:])
    c = ref.Batch(_rng(33), 8, 1, 128, 64, "bf16", seqs)
    c.seqs = seqs[:2] + [(2, 2 ** 31 - 1)] + seqs[3:]  # past its table
    assert c.call(window=150, sinks=4) == smq.SMQ_ERR_BOUNDS
    c.check([sets[0], sets[1], [np.arange(4)] * 2, sets[3]])
    for cu in ([0, 3, 2, 13, 17], [0, 3, 11, 13, 400], [-1, 3, 11, 13, 17]):
        c = ref.Batch(_rng(34), 8, 1, 128, 64, "bf16", seqs)
        c.cu = np.array(cu, np.int32)
        assert c.call(window=150, sinks=4, max_seq_rows=11) & smq.SMQ_ERR_BOUNDS


def test_a_cache_past_32_bits():
    """Pages whose element offsets pass 2^32."""
    page, dim = 64, 128
    pages = 2 ** 32 // (2 * page * dim) + 40
    plan = smq.AttentionPlan(16, 1, dim, page, max_rows=4)
    data = torch.empty(pages, 2, 1, page, dim, device=DEV, dtype=torch.bfloat16)
    table = torch.tensor([[pages - 1, 0, pages - 20], [pages // 2 + 1, pages - 2, 1]], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for row in table.tolist():
        for p in row:
            data[p] = torch.randn(2, 1, page, dim, generator=g, device=DEV)
    q = torch.randn(4, 16, dim, generator=g, device=DEV).to(torch.bfloat16)
    out, lse, ws = torch.empty_like(q), torch.empty(4, 16, device=DEV), plan.sequence_workspace()
    smq.sparse_mqa_attention_window(plan, q, data[:, 0], data[:, 1], table, torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV),
                                    torch.tensor([180, 192], dtype=torch.int32, device=DEV), 2, out, ws, 1000, lse=lse)
    assert smq.smq_get_status(ws) == 0
    for r, (s, n) in enumerate(((0, 179), (0, 180), (1, 191), (1, 192))):
        both = data[table[s].long()].cpu().to(torch.float64).numpy()
        k, v = (both[:, side].transpose(0, 2, 1, 3).reshape(-1, 1, dim)[:n] for side in (0, 1))
        want, mean, want_lse, size = ref.attend(q[r].cpu().to(torch.float64).numpy(), k, v, dim ** -0.5)
        off, lse_off = ref.bound(want, mean, size, dim, n)
        assert (np.abs(out[r].cpu().to(torch.float64).numpy() - want) <= off).all()
        assert (np.abs(lse[r].cpu().to(torch.float64).numpy() - want_lse) <= lse_off + 2.0 ** -22 * np.abs(want_lse)).all()


def test_streams_and_graphs():
    """Calls on a stream of their own, and replayed from a graph on lengths that changed in place; two workspaces at once."""
    rng = _rng(21)
    seqs = [(4, 3000), (30, 200), (1, 77)]
    b = ref.Batch(rng, 16, 1, 128, 64, "bf16", seqs)
    assert b.call(window=1, sinks=0) == 0
    sets = [ref.window_sets(n, length, 900, 4) for n, length in seqs]
    args = dict(b.cache.to(DEV), block_table=torch.from_numpy(b.table).to(DEV), cu_rows=torch.from_numpy(b.cu).to(DEV),
                seq_indices=torch.from_numpy(b.order).to(DEV), max_seq_rows=30, window=900, sinks=4)
    length = torch.tensor([4, 30, 1], dtype=torch.int32, device=DEV)
    outs = [(torch.full_like(b.out, 9), torch.full_like(b.lse, 9)) for _ in range(2)]
    calls = [smq.SequenceAttentionCall(b.plan, b.q_dev, seq_len=length, out=o, lse=x, workspace=b.plan.sequence_workspace(), **args)
             for o, x in outs]
    side = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for s, call in zip(side, calls):
        with torch.cuda.stream(s):
            call()
    torch.cuda.synchronize()
    for b.out, b.lse in outs:
        b.check([ref.window_sets(n, n, 900, 4) for n, _ in seqs])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls[0]()
        calls[1]()
    length.copy_(torch.tensor([n for _, n in seqs], dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(smq.smq_get_status(c._keep[7]) == 0 for c in calls)
    for b.out, b.lse in outs:
        b.check(sets)


def test_no_rows_and_no_sequences():
    plan = smq.AttentionPlan(4, 2, 64, 16, max_rows=4)
    data = torch.zeros(2, 2, 2, 16, 64, device=DEV, dtype=torch.bfloat16)
    ws = plan.sequence_workspace()
    for rows, seqs in ((0, 2), (3, 0), (0, 0)):
        q = torch.zeros(rows, 4, 64, device=DEV, dtype=torch.bfloat16)
        out = torch.full_like(q, 5)
        cu = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
        table = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
        smq.sparse_mqa_attention_window(plan, q, data[:, 0], data[:, 1], table, cu, cu[:seqs].clone(), 1, out, ws, 5)
        smq.sparse_mqa_attention_tree(plan, q, data[:, 0], data[:, 1], table, cu, cu[:seqs].clone(), 1, out, ws,
                                      torch.zeros(rows, 1, dtype=torch.int32, device=DEV))
        assert smq.smq_get_status(ws) == 0 and (out == 5).all()


# ------------------------------------------------------------------ refusals


def _tensors(tree, rows=3):
    data = torch.zeros(4, 2, 2, 16, 64, device=DEV, dtype=torch.bfloat16)
    plan = smq.AttentionPlan(8, 2, 64, 16, max_rows=4)
    q = torch.zeros(rows, 8, 64, device=DEV, dtype=torch.bfloat16)
    args = dict(k_cache=data[:, 0], v_cache=data[:, 1], block_table=torch.zeros(4, 4, dtype=torch.int32, device=DEV),
                cu_rows=torch.tensor([0, 1, rows], dtype=torch.int32, device=DEV),
                seq_len=torch.tensor([5, 5], dtype=torch.int32, device=DEV), max_seq_rows=3, out=torch.empty_like(q),
                workspace=plan.sequence_workspace())
    args.update(dict(tree_mask=torch.zeros(rows, 1, dtype=torch.int32, device=DEV)) if tree else dict(window=4, sinks=1))
    return plan, q, args


BAD = smq.SMQ_ERR_INVALID_ARG


@pytest.mark.parametrize("tree,field,value,code", [
    (False, "rows", 5, BAD), (False, "rows", -1, BAD), (False, "num_seqs", 5, BAD), (False, "num_seqs", -1, BAD),
    (False, "max_seq_rows", 0, BAD), (False, "max_seq_rows", 5, BAD), (False, "window", 0, BAD), (False, "window", -3, BAD),
    (False, "sinks", -1, BAD), (False, "mask_words", 1, BAD), (False, "q", None, BAD), (False, "q_stride", 4, BAD),
    (False, "q_stride", 8 * 64 + 4, BAD), (False, "k_cache", None, BAD), (False, "num_pages", 0, BAD),
    (False, "page_stride", 16, BAD), (False, "block_table", None, BAD), (False, "cu_rows", None, BAD),
    (False, "seq_len", None, BAD), (False, "out", None, BAD), (False, "workspace", None, BAD),
    (False, "workspace_bytes", 128, smq.SMQ_ERR_WORKSPACE_TOO_SMALL), (False, "struct_size", 16, BAD),
    (True, "tree_mask", None, BAD), (True, "mask_words", 0, BAD), (True, "mask_words", 33, BAD), (True, "window", 4, BAD),
    (True, "sinks", 1, BAD), (True, "seq_len", None, BAD), (True, "struct_size", 16, BAD),
])
def test_the_library_refuses_bad_arguments(tree, field, value, code):
    plan, q, args = _tensors(tree)
    call = smq.SequenceAttentionCall(plan, q, **args)
    setattr(call.args, field, value)
    with pytest.raises(smq.SMQError) as e:
        call()
    assert e.value.code == code
    assert smq.smq_get_status(args["workspace"]) == 0


def test_more_rows_than_mask_bits_are_refused():
    plan = smq.AttentionPlan(8, 2, 64, 16, max_rows=64)
    _, q, args = _tensors(True)
    args["max_seq_rows"] = 33
    with pytest.raises(smq.SMQError) as e:
        smq.SequenceAttentionCall(plan, q, **args)()
    assert e.value.code == BAD


@pytest.mark.parametrize("change,error", [
    (dict(window=None), ValueError), (dict(tree_mask="both"), ValueError), (dict(cu_rows="short"), ValueError),
    (dict(seq_len="cpu"), ValueError), (dict(seq_len="long"), TypeError), (dict(block_table="short"), ValueError),
    (dict(out="short"), ValueError), (dict(lse="short"), ValueError), (dict(k_scales="extra"), ValueError),
])
def test_the_binding_refuses_what_does_not_fit(change, error):
    plan, q, args = _tensors(False)
    (name, what), = change.items()
    if what is None:
        args[name] = None
    elif what == "both":
        args[name] = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    elif what == "cpu":
        args[name] = args[name].cpu()
    elif what == "long":
        args[name] = args[name].long()
    elif what == "extra":
        args[name] = torch.ones(4, 2, 16, device=DEV)
    elif name == "lse":
        args[name] = torch.zeros(2, 8, device=DEV)
    else:
        args[name] = args[name][:1]
    with pytest.raises(error):
        smq.SequenceAttentionCall(plan, q, **args)
