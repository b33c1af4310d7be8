"""The sequences' attention at the ends of its ranges: more rows than a call of single rows takes, as many sequences, and one
prefill of them all."""

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


def _sets(seqs, window, sinks):
    """What ref.window_sets says, by ranges: the contexts here are long."""
    got = []
    for n, length in seqs:
        per = []
        for at in range(length - n, length):
            lo = max(0, at + 1 - window)
            per.append(np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, max(0, at + 1))]).astype(np.int64))
        got.append(per)
    return got


def test_the_sets_are_those_of_the_plain_form():
    for n, length, window, sinks in ((3, 6, 2, 1), (3, 2, 5, 0), (9, 40, 7, 12), (5, 5, 1, 2)):
        want = ref.window_sets(n, length, window, sinks)
        assert [x.tolist() for x in _sets([(n, length)], window, sinks)[0]] == [x.tolist() for x in want]


@pytest.mark.parametrize("heads,kv_heads,dtype,seqs", [
    (8, 1, "bf16", [(213 + 40 * i // 59, 213 + 40 * i // 59 + 10 * i) for i in range(60)]),  # ragged chunks, 13954 rows with padding
    (4, 2, "e4m3", [(9001, 9300), (1, 50)]),                                                 # one long prefill
    (2, 1, "bf16", [(1, 1 + i % 90) for i in range(9500)]),                                  # a token of each of many sequences
])
def test_more_rows_than_a_call_of_single_rows(heads, kv_heads, dtype, seqs):
    b = ref.Batch(_rng(heads, len(seqs)), heads, kv_heads, 64, 64, dtype, seqs)
    assert b.rows > smq.AttentionPlan.MAX_SINGLE_ROWS and b.plan.max_rows == b.rows
    assert b.call(window=300, sinks=3) == 0
    sets = _sets(seqs, 300, 3)
    b.check(sets, rows={i for n, _ in seqs[:70] for i in range(n) if i < 3 or i % 97 == 0 or i > n - 4})
    if max(n for n, _ in seqs) == 1:
        b.tree([{0}] * len(seqs))


def test_an_append_of_as_many_rows():
    rows, page, pages = 9000, 64, 150
    plan = smq.AttentionPlan(4, 2, 64, page, max_rows=rows)
    data = torch.zeros(pages, 2, 2, page, 64, device=DEV, dtype=torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(rows, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:rows]
    ws = plan.workspace()
    smq.sparse_mqa_append_kv(plan, None, k, v, None, None, slots, data[:, 0], data[:, 1], ws)
    assert smq.smq_get_status(ws) == 0
    for side, x in ((0, k), (1, v)):
        assert torch.equal(data[slots // page, side, :, slots % page], x)


def test_calls_of_single_rows_keep_their_bound():
    rows = smq.AttentionPlan.MAX_SINGLE_ROWS + 1
    plan = smq.AttentionPlan(1, 1, 64, 16, max_rows=rows)
    data = torch.zeros(2, 2, 1, 16, 64, device=DEV, dtype=torch.bfloat16)
    q = torch.zeros(rows, 1, 64, device=DEV, dtype=torch.bfloat16)
    out, table = torch.full_like(q, 5), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ws, at = plan.workspace(), torch.zeros(rows, dtype=torch.int32, device=DEV)
    with pytest.raises(smq.SMQError) as e:
        smq.sparse_mqa_attention_decode(plan, q, data[:, 0], data[:, 1], table, at, at + 1, out, ws)
    assert e.value.code == smq.SMQ_ERR_INVALID_ARG and (out == 5).all()
    smq.sparse_mqa_attention_decode(plan, q[1:], data[:, 0], data[:, 1], table, at[1:], at[1:] + 1, out[1:], ws)
    assert smq.smq_get_status(ws) == 0 and (out[1:] == 0).all() and (out[0] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (128, 1)])
def test_drafted_tokens_past_the_table(dtype, heads, kv_heads):
    """A drafted token without a place in the table is an error only where a row's mask has it, or has its position."""
    page, columns, n = 16, 5, 40
    top = page * columns
    for length, bits, status in (
            (top + 3, lambda i: {j for j in range(37) if j <= i}, 0),                # nodes 37 to 39 are seen by nobody
            (top + 3, lambda i: {0, 5} | {40, 50, 63}, 0),                           # bits past the rows are not read
            (top + 3, lambda i: {36, 37} if i == 33 else {36}, smq.SMQ_ERR_BOUNDS),  # one row sees one
            (top + 39, lambda i: {0}, 0), (top + 39, lambda i: {1}, smq.SMQ_ERR_BOUNDS),
            (top + 40, lambda i: set(), 0),                                          # the context ends with the table
            (top + 41, lambda i: set(), smq.SMQ_ERR_BOUNDS)):                        # every row sees a token past it
        masks = [bits(i) for i in range(n)]
        b = ref.Batch(_rng(length), heads, kv_heads, 64, page, dtype, [(3, 20), (n, top)])
        b.seqs = [(3, 20), (n, length)]
        packed = ref.pack([{0}] * 3 + masks + [set()] * 2, 2)
        assert b.call(tree_mask=packed) == status, length
        sets = [ref.tree_sets(3, 20, [{0}] * 3), [s[s < top] for s in ref.tree_sets(n, length, masks)]]
        b.check(sets)


@pytest.mark.parametrize("length", [2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 5, 2 ** 31 - 1])
@pytest.mark.parametrize("max_seq_rows", [1, 200])
def test_the_longest_contexts(length, max_seq_rows):
    """Every token has the same score. The first page's values are -1, all others' are one page's, 1, so a result that counts every
    token is 1 - 2 * 65536 / length, 1 in bf16; sums of ones are exact in fp32 up to 2^24, and a CTA's are 2^24 at most."""
    page, columns = 65536, 32768
    plan = smq.AttentionPlan(1, 1, 64, page, max_rows=200)
    data = torch.zeros(2, 2, 1, page, 64, device=DEV, dtype=torch.bfloat16)
    data[0, 1], data[1, 1] = -1, 1
    table = torch.ones(1, columns, dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    q = torch.ones(1, 1, 64, device=DEV, dtype=torch.bfloat16)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1], [length]))
    ws = plan.sequence_workspace()
    for what in (dict(window=2 ** 31 - 1), dict(tree_mask=torch.ones(1, 1, dtype=torch.int32, device=DEV))):
        if max_seq_rows > 32 and "tree_mask" in what:
            what["tree_mask"] = torch.ones(1, 7, dtype=torch.int32, device=DEV)
        out, lse = torch.zeros_like(q), torch.zeros(1, 1, device=DEV)
        smq.SequenceAttentionCall(plan, q, data[:, 0], data[:, 1], table, cu, lens, max_seq_rows, out, ws, lse=lse, **what)()
        assert smq.smq_get_status(ws) == 0
        assert (out == 1).all() and abs(float(lse) - np.log(float(length))) < 1e-5


def test_a_window_at_the_end_of_the_longest_context():
    """The newest rows of a context of 2^31 - 1 tokens, whose pages before the window are gone."""
    page, columns = 65536, 32768
    plan = smq.AttentionPlan(2, 1, 64, page, max_rows=200)
    g = torch.Generator(device=DEV).manual_seed(2)
    data = torch.randn(3, 2, 1, page, 64, generator=g, device=DEV).to(torch.bfloat16)
    table = torch.full((1, columns), -1, dtype=torch.int32, device=DEV)
    table[0, 0], table[0, -1], table[0, -2] = 2, 0, 1
    rows, length, window, sinks = 150, 2 ** 31 - 1, 70000, 3
    q = torch.randn(rows, 2, 64, generator=g, device=DEV).to(torch.bfloat16)
    out, lse, ws = torch.zeros_like(q), torch.zeros(rows, 2, device=DEV), plan.sequence_workspace()
    cu, lens = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, rows], [length]))
    smq.sparse_mqa_attention_window(plan, q, data[:, 0], data[:, 1], table, cu, lens, rows, out, ws, window, sinks, lse=lse)
    assert smq.smq_get_status(ws) == 0
    both = torch.cat([data[2, :, 0, :sinks], data[1, :, 0], data[0, :, 0]], 1).double().cpu().numpy()  # sinks, the last two pages
    for r in (0, 1, 77, 149):
        at = length - rows + r  # position; the last two pages begin at (columns - 2) * page
        hi = at + 1 - (columns - 2) * page
        seen = np.r_[0:sinks, sinks + hi - window:sinks + hi]
        k, v = both[0][seen][:, None], both[1][seen][:, None]
        want, mean, want_lse, size = ref.attend(q[r].double().cpu().numpy(), k, v, 0.125)
        off, lse_off = ref.bound(want, mean, size, 64, len(seen))
        assert (np.abs(out[r].double().cpu().numpy() - want) <= off).all(), r
        assert (np.abs(lse[r].double().cpu().numpy() - want_lse) <= lse_off + 2.0 ** -22 * np.abs(want_lse)).all(), r


@pytest.mark.parametrize("heads,kv_heads,dtype", [(64, 8, "bf16"), (3, 1, "bf16"), (16, 2, "e4m3"), (128, 1, "e4m3")])
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("top", [1e5, 3e8, 1e10, 1e20, 2.2e38])
def test_scores_far_from_zero(heads, kv_heads, dtype, scale, top):
    """Scores up to `top` in steps of an eighth of it, of either sign, many of them equal: the largest share all the weight. Their
    roundings do not matter, as equal scores round alike and others are far off; lse has seven, of products, scales and sums,
    2^-24 of it each."""
    if dtype == "e4m3":  # a product is of a query and a code, 448 here, before the token's scale: 56 * top, which has to be finite
        top = min(top, 5e36)
    rng = _rng(heads, int(np.log10(top)))
    seqs = [(1, 1), (2, 130), (40, 400), (1, 3000), (3, 5)]
    b = ref.Batch(rng, heads, kv_heads, 128, 64, dtype, seqs, scale=scale)
    b.q[:] = 0
    strength = torch.from_numpy(rng.choice([-1.0, 1.0, 0.3], b.q.shape[:2]) * top / 8).to(torch.bfloat16)
    b.q[:, :, 3] = strength
    for i, (_, n) in enumerate(seqs):
        keys = np.zeros((n, kv_heads, 128))
        keys[:, :, 3] = rng.integers(1, 9, (n, kv_heads)) * rng.choice([-1, 1], (1, kv_heads))  # of one sign: all scores far off, or none
        bounds.put(b.cache, i, np.arange(n), 0, keys)
    sets = _sets(seqs, 1500, 4)
    assert b.call(sets, window=1500, sinks=4) == 0
    out, lse = b.out.double().cpu().numpy(), b.lse.double().cpu().numpy()
    for i, per in enumerate(sets):
        for r, at in zip(range(b.cu[i], b.cu[i + 1]), per):
            k, v = b.cache.tokens(i, at)
            want, mean, want_lse, _ = ref.attend(b.q[r].double().numpy(), k, v, scale)
            off, lse_off = ref.bound(want, mean, np.zeros(heads), 128, len(at))
            assert (np.abs(out[r] - want) <= off).all(), (i, r)
            assert (np.abs(lse[r] - want_lse) <= lse_off + 2.0 ** -21 * np.abs(want_lse)).all(), (i, r)


@pytest.mark.parametrize("name", ["window", "sinks", "max_seq_rows", "keep_first"])
def test_numbers_past_32_bits_are_refused(name):
    """A window of 2^32 + 4 tokens is not one of 4."""
    plan = smq.AttentionPlan(4, 2, 64, 16, max_rows=4)
    data = torch.zeros(2, 2, 2, 16, 64, device=DEV, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 64, device=DEV, dtype=torch.bfloat16)
    table, cu, n = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([[0]], [0, 1], [5]))
    what = dict(window=4, sinks=0, max_seq_rows=1)
    with pytest.raises(ValueError, match="32 bits"):
        if name == "keep_first":
            pool = smq.PagePlan(16, 4, 1, 2)
            refs, state = pool.state()
            smq.ResizeCall(pool, refs, state, n, pool.workspace(), keep_first=2 ** 32)
        else:
            smq.SequenceAttentionCall(plan, q, data[:, 0], data[:, 1], table, cu, n, out=torch.empty_like(q),
                                      workspace=plan.sequence_workspace(), **{**what, name: 2 ** 32 + 4})


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 60])
def test_a_wait_limit_of_a_nanosecond(dtype, rows):
    """The clock is looked at every sixteenth try of a wait, each of which the hardware may hold up until the phase is there, so a call
    in which nothing is late may end without an error; one with a tile that is never handed over may not. The next is right."""
    seqs = [(rows, 2000 + 60 * i) for i in range(6)]
    b = ref.Batch(_rng(rows), 64, 8, 128, 64, dtype, seqs)
    sets = _sets(seqs, 1500, 4)
    b.plan.set_wait_limit(1)
    assert all(b.call(window=1500, sinks=4) in (0, smq.SMQ_ERR_TIMEOUT) for _ in range(5))
    b.plan.inject_stall(1)
    for _ in range(5):
        assert b.call(window=1500, sinks=4) == smq.SMQ_ERR_TIMEOUT
        b.plan.inject_stall(-1)
        b.plan.set_wait_limit(2_000_000_000)
        assert b.call(window=1500, sinks=4) == 0
        b.plan.inject_stall(1)
        b.plan.set_wait_limit(1)
    b.plan.inject_stall(-1)
    b.plan.set_wait_limit(2_000_000_000)
    assert b.call(window=1500, sinks=4) == 0
    b.check(sets, rows={0, rows - 1})
