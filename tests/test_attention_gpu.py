"""The attention operators against plain 64-bit forms, through the public entry points: appending rotated keys and
values, attention over a cached range, attention over selected token ids."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def _check(got, lse, want, dtype, where):
    out, ref_lse, mean, top, total = want
    got = got.to(torch.float64).cpu().numpy()
    lse = lse.to(torch.float64).cpu().numpy()
    off = np.abs(got - out) - ref.tolerance(out, mean, top, total, dtype)
    assert np.isfinite(got).all(), f"{where}: not finite"
    assert (off <= 0).all(), f"{where}: over the tolerance by {off.max():.3g} at {np.argwhere(off > 0)[:3].tolist()}"
    empty = np.isinf(ref_lse)
    assert np.array_equal(lse[empty], ref_lse[empty]), f"{where}: lse of an empty row"
    assert (np.abs(lse - ref_lse)[~empty] <= 5e-4 + 1e-6 * np.abs(ref_lse[~empty])).all(), f"{where}: lse"


# ------------------------------------------------------------------- append


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype,rot,interleaved,rows", [
    (64, 8, 128, 64, "bf16", 128, False, 37),
    (64, 1, 128, 64, "bf16", 64, True, 1),
    (6, 3, 64, 16, "bf16", 32, False, 130),
    (8, 2, 64, 7, "bf16", 0, False, 19),
    (64, 8, 128, 64, "e4m3", 128, False, 65),
    (20, 4, 64, 32, "e4m3", 64, True, 33),
    (3, 1, 128, 1, "e4m3", 16, True, 5),
    (64, 8, 128, 64, "e4m3", 128, False, 2500),
])
def test_append_matches_bit_for_bit(heads, kv_heads, dim, page, dtype, rot, interleaved, rows):
    rng = np.random.Generator(np.random.PCG64(7 + rows))
    positions = 50
    angle = rng.standard_normal((positions, max(rot // 2, 1))) * 100
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = rng.integers(0, positions, rows)
    pages = -(-rows // page) + 2
    slots = rng.permutation(pages * page)[:rows]
    slots[rng.random(rows) < 0.1] = -1
    x = rng.standard_normal((rows, (heads + 2 * kv_heads) * dim)).astype(np.float32)
    x *= np.exp(rng.standard_normal((rows, 1)) * 3).astype(np.float32)
    x[rows // 2, heads * dim:] = 0  # zero keys and values: scale 1
    qkv = _bf16(x)
    xf = qkv.to(torch.float32).numpy()
    q, k, v = (a.reshape(rows, -1, dim) for a in np.split(xf, [heads * dim, (heads + kv_heads) * dim], 1))
    if rot:
        half = rot // 2
        c, s = cos_sin[pos, :half], cos_sin[pos, half:]
        q, k = ref.rotate(q, c, s, interleaved), ref.rotate(k, c, s, interleaved)
    plan = smq.AttentionPlan(heads, kv_heads, dim, page, max_rows=rows, cache_dtype=dtype)
    dev = qkv.to(DEV)
    q_out = torch.full((rows, heads, dim), 7.0, device=DEV, dtype=torch.bfloat16)
    data = torch.full((pages, 2, kv_heads, page, dim), 3, device=DEV, dtype=torch.bfloat16 if dtype == "bf16" else torch.uint8)
    scales = None if dtype == "bf16" else torch.full((pages, 2, kv_heads, page), 5.0, device=DEV)
    want, want_scales = data.cpu().clone(), None if scales is None else scales.cpu().clone()
    for t in range(rows):
        if slots[t] < 0:
            continue
        at = slots[t] // page, slots[t] % page
        for side, y in ((0, k[t]), (1, v[t])):
            if dtype == "bf16":
                want[at[0], side, :, at[1]] = _bf16(y)
            else:
                code, scale = ref.quantise(y)
                want[at[0], side, :, at[1]] = torch.from_numpy(code)
                want_scales[at[0], side, :, at[1]] = torch.from_numpy(scale)
    ws = plan.workspace()
    smq.sparse_mqa_append_kv(
        plan, dev[:, :heads * dim].view(rows, heads, dim),
        dev[:, heads * dim:(heads + kv_heads) * dim].view(rows, kv_heads, dim),
        dev[:, (heads + kv_heads) * dim:].view(rows, kv_heads, dim),
        torch.from_numpy(pos).to(DEV) if rot else None, torch.from_numpy(cos_sin).to(DEV) if rot else None,
        torch.from_numpy(slots).to(DEV), data[:, 0], data[:, 1], ws, q_out=q_out,
        k_scales=None if scales is None else scales[:, 0], v_scales=None if scales is None else scales[:, 1],
        interleaved=interleaved)
    assert smq.smq_get_status(ws) == 0
    assert torch.equal(q_out.cpu().view(torch.int16), _bf16(q).view(torch.int16)), "queries"
    bits = torch.int16 if dtype == "bf16" else torch.uint8
    assert torch.equal(data.cpu().view(bits), want.view(bits)), "cache"
    if scales is not None:
        assert torch.equal(scales.cpu(), want_scales), "scales"


def test_append_reports_what_is_out_of_range():
    plan = smq.AttentionPlan(4, 2, 64, 16, max_rows=4)
    x = torch.randn(4, 4, 64, device=DEV, dtype=torch.bfloat16)
    table = torch.ones(10, 64, device=DEV)
    for pos, slots, written in (([0, 1, 10, 3], [0, 1, 2, 3], [0, 1, 3]), ([0, 1, 2, -1], [0, 1, 2, 3], [0, 1, 2]),
                                ([0, 1, 2, 3], [0, 32, 2, 3], [0, 2, 3])):
        data = torch.zeros(2, 2, 2, 16, 64, device=DEV, dtype=torch.bfloat16)
        ws = plan.workspace()
        smq.sparse_mqa_append_kv(plan, None, x[:, :2].contiguous(), x[:, 2:].contiguous(),
                                 torch.tensor(pos, device=DEV), table, torch.tensor(slots, device=DEV), data[:, 0],
                                 data[:, 1], ws)
        assert smq.smq_get_status(ws) == smq.SMQ_ERR_BOUNDS
        assert smq.smq_get_status(ws) == 0, "reading clears the status"
        got = torch.nonzero(data[:, 1].abs().sum((1, 3)).flatten()).flatten().tolist()
        assert got == written, "the other tokens are written"


# ---------------------------------------------------------------- attention


class Rows:
    """Query rows over a Cache, and the outputs of a call."""

    def __init__(self, rng, cache, heads, seqs, max_rows=None, scale=None):
        self.cache, self.seqs = cache, seqs
        rows = len(seqs)
        wide = _bf16(rng.standard_normal((rows, heads * cache.dim + 8)) * 1.5)  # rows a stride apart
        self.q = wide[:, :heads * cache.dim].view(rows, heads, cache.dim)
        self.plan = smq.AttentionPlan(heads, cache.kv_heads, cache.dim, cache.page, max_rows=max_rows or rows,
                                      cache_dtype=cache.dtype, softmax_scale=scale)
        self.scale = scale or 1 / math.sqrt(cache.dim)
        self.dev = dict(cache.to(DEV), block_table=torch.from_numpy(cache.table).to(DEV),
                        row_indices=torch.tensor(seqs, dtype=torch.int32, device=DEV),
                        out=torch.full((rows, heads, cache.dim), 9.0, device=DEV, dtype=torch.bfloat16),
                        lse=torch.full((rows, heads), 9.0, device=DEV), workspace=self.plan.workspace())
        self.q_dev = wide.to(DEV)[:, :heads * cache.dim].view(rows, heads, cache.dim)

    def call(self, **kw):
        smq.AttentionCall(self.plan, self.q_dev, **self.dev, **kw)()
        return smq.smq_get_status(self.dev["workspace"])

    def check(self, positions, rows=None):
        q = self.q.to(torch.float64).numpy()
        for r in range(len(self.seqs)) if rows is None else rows:
            k, v = self.cache.tokens(self.seqs[r], positions[r])
            _check(self.dev["out"][r], self.dev["lse"][r], ref.attend(q[r], k, v, self.scale), self.cache.dtype, f"row {r}")


GEOMETRIES = [  # heads, kv heads, dim, page, dtype: every padded group size and odd groups of it
    (1, 1, 128, 64, "bf16"), (8, 8, 128, 64, "bf16"), (16, 1, 128, 16, "bf16"), (64, 8, 64, 64, "bf16"),
    (24, 1, 64, 32, "bf16"), (64, 2, 128, 64, "bf16"), (64, 1, 128, 64, "bf16"), (33, 1, 64, 5, "bf16"),
    (128, 1, 128, 64, "bf16"), (130, 2, 64, 128, "bf16"),
    (1, 1, 128, 64, "e4m3"), (24, 3, 64, 16, "e4m3"), (64, 2, 64, 64, "e4m3"), (64, 1, 128, 64, "e4m3"),
    (41, 1, 64, 32, "e4m3"), (128, 1, 128, 64, "e4m3"), (66, 1, 64, 9, "e4m3"),
]


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
def test_decode_matches(heads, kv_heads, dim, page, dtype):
    rng = np.random.Generator(np.random.PCG64(heads + dim))
    lens = [0, 1, 2, 127, 128, 129, 255, 256, 300, 1000, 64, 700]
    cache = ref.Cache(rng, kv_heads, dim, page, dtype, lens)
    seqs = [int(i) for i in rng.permutation(len(lens))] + [9, 0, 9]
    rows = Rows(rng, cache, heads, seqs)
    ke = [lens[s] for s in seqs]
    assert rows.call(row_ke=torch.tensor(ke, dtype=torch.int32, device=DEV)) == 0
    rows.check([np.arange(n) for n in ke])


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
def test_selected_matches(heads, kv_heads, dim, page, dtype):
    rng = np.random.Generator(np.random.PCG64(heads + 3 * dim))
    lens = [700, 1, 300, 40]
    cache = ref.Cache(rng, kv_heads, dim, page, dtype, lens)
    seqs = [0, 1, 2, 3, 0, 0, 2, 0]
    num = 413
    ids = np.full((len(seqs), num), -1, np.int32)
    for r, s in enumerate(seqs):
        n = min(num, lens[s])
        ids[r, :n] = rng.permutation(lens[s])[:n]
    ids[4, :] = -1                                 # no token at all
    ids[5] = np.where(rng.random(num) < 0.6, -1, ids[5])  # holes
    ids[6, 1:] = ids[6, 0]                         # one token many times
    ids[7, :400] = -1                              # only the end of the list
    rows = Rows(rng, cache, heads, seqs)
    assert rows.call(token_ids=torch.from_numpy(ids).to(DEV)) == 0
    rows.check([i[i >= 0] for i in ids])


@pytest.mark.parametrize("num", [1, 64, 128, 129])
def test_selected_lists_of_few_ids(num):
    rng = np.random.Generator(np.random.PCG64(num))
    cache = ref.Cache(rng, 1, 128, 64, "bf16", [200] * 3)
    ids = np.stack([rng.permutation(200)[:num] for _ in range(3)]).astype(np.int32)
    rows = Rows(rng, cache, 8, [2, 0, 1])
    assert rows.call(token_ids=torch.from_numpy(ids).to(DEV)) == 0
    rows.check(ids)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_of_a_window(dtype):
    """row_ks cuts the start of the range, also inside a page and a tile, and past the end."""
    rng = np.random.Generator(np.random.PCG64(5))
    lens = [500] * 6
    cache = ref.Cache(rng, 2, 128, 64, dtype, lens)
    ks, ke = [0, 3, 130, 499, 500, 450], [500, 260, 500, 500, 500, 400]
    rows = Rows(rng, cache, 32, list(range(6)))
    assert rows.call(row_ke=torch.tensor(ke, dtype=torch.int32, device=DEV),
                     row_ks=torch.tensor(ks, dtype=torch.int32, device=DEV)) == 0
    rows.check([np.arange(a, b) for a, b in zip(ks, ke)])


@pytest.mark.parametrize("heads,kv_heads,dtype,lens", [
    (8, 1, "bf16", [60001]),                 # one row over every CTA
    (64, 1, "e4m3", [20000, 3, 0, 9000]),    # a row over many CTAs beside tiny ones
    (16, 4, "bf16", [5000, 12345, 1]),
])
def test_rows_split_over_ctas(heads, kv_heads, dtype, lens):
    rng = np.random.Generator(np.random.PCG64(len(lens)))
    cache = ref.Cache(rng, kv_heads, 128, 64, dtype, lens)
    rows = Rows(rng, cache, heads, list(range(len(lens))))
    ke = torch.tensor(lens, dtype=torch.int32, device=DEV)
    assert rows.call(row_ke=ke) == 0
    rows.check([np.arange(n) for n in lens])
    first = rows.dev["out"].clone(), rows.dev["lse"].clone()
    assert rows.call(row_ke=ke) == 0
    assert torch.equal(first[0], rows.dev["out"]) and torch.equal(first[1], rows.dev["lse"]), "the same bits again"


def test_many_rows_of_several_tiles():
    """More rows than threads of a CTA, lengths from none to several tiles."""
    rng = np.random.Generator(np.random.PCG64(77))
    lens = [0, 1, 130, 400, 260, 128]
    cache = ref.Cache(rng, 1, 64, 16, "bf16", lens)
    seqs = [int(s) for s in rng.integers(0, len(lens), 1300)]
    rows = Rows(rng, cache, 4, seqs)
    ke = [lens[s] for s in seqs]
    assert rows.call(row_ke=torch.tensor(ke, dtype=torch.int32, device=DEV)) == 0
    rows.check([np.arange(n) for n in ke], rows=range(0, 1300, 13))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("growth", [1.0, -1.0])
def test_scores_that_rise_and_fall(dtype, growth):
    """Large scores, growing or shrinking along the row: the running maximum moves many times, or never again."""
    rng = np.random.Generator(np.random.PCG64(15))
    cache = ref.Cache(rng, 1, 128, 64, dtype, [1500])
    rows = Rows(rng, cache, 40, [0])
    # keys lean towards one direction, more and more; the queries follow it with strengths of both signs
    lean = np.linspace(0, 1, 1500)[::int(growth)]
    d = np.zeros(128)
    d[5] = 1
    for p in range(1500):
        page, off = cache.table[0][p // 64], p % 64
        key = cache.values[page, 0, 0, off] * 0.3 + 12 * lean[p] * d
        if dtype == "bf16":
            cache.data[page, 0, 0, off] = _bf16(key)
            cache.values[page, 0, 0, off] = _bf16(key).to(torch.float64).numpy()
        else:
            code, scale = ref.quantise(key.astype(np.float32))
            cache.data[page, 0, 0, off] = torch.from_numpy(code)
            cache.scales[page, 0, 0, off] = float(scale)
            cache.values[page, 0, 0, off] = ref.e4m3_values(code) * np.float64(scale)
    q = rows.q.clone()
    q[0, :, 5] = torch.linspace(-60, 60, 40).to(torch.bfloat16)
    rows.q = q
    rows.q_dev = q.to(DEV)
    rows.dev.update(cache.to(DEV))
    assert rows.call(row_ke=torch.tensor([1500], dtype=torch.int32, device=DEV)) == 0
    rows.check([np.arange(1500)])


def test_softmax_scale_and_identity_rows():
    rng = np.random.Generator(np.random.PCG64(8))
    lens = [150, 33, 260]
    cache = ref.Cache(rng, 2, 64, 64, "bf16", lens)
    rows = Rows(rng, cache, 8, [0, 1, 2], scale=-0.31)
    rows.dev["row_indices"] = None
    assert rows.call(row_ke=torch.tensor(lens, dtype=torch.int32, device=DEV)) == 0
    rows.check([np.arange(n) for n in lens])


def test_out_of_range_pages_and_positions_are_left_out():
    rng = np.random.Generator(np.random.PCG64(9))
    lens = [300, 300, 300, 300]
    cache = ref.Cache(rng, 1, 128, 64, "bf16", lens)
    rows = Rows(rng, cache, 16, [0, 1, 2, 3, 4])   # row 4: no such table row
    table = cache.table.copy()
    table[1, 1] = -5
    table[2, 3] = cache.pages
    rows.dev["block_table"] = torch.from_numpy(table).to(DEV)
    ke = torch.tensor([300, 300, 300, 2 ** 31 - 1, 300], dtype=torch.int32, device=DEV)  # row 3: past its table
    assert rows.call(row_ke=ke) == smq.SMQ_ERR_BOUNDS
    keep = [np.arange(300), np.r_[0:64, 128:300], np.r_[0:192, 256:300]]
    rows.check(keep, rows=range(3))
    assert bool((rows.dev["out"][4] == 0).all())
    ids = np.array([[0, 299, 320, 7]] * 5, np.int32)   # 320: past the table's five pages
    assert rows.call(token_ids=torch.from_numpy(ids).to(DEV)) == smq.SMQ_ERR_BOUNDS
    rows.check([[0, 299, 7]], rows=[0])


def test_a_cache_past_32_bits():
    """Pages whose element offsets pass 2^32."""
    page, dim = 64, 128
    pages = 2 ** 32 // (2 * page * dim) + 40
    plan = smq.AttentionPlan(16, 1, dim, page, max_rows=2)
    data = torch.empty(pages, 2, 1, page, dim, device=DEV, dtype=torch.bfloat16)
    table = torch.tensor([[pages - 1, 0, pages - 20], [pages // 2 + 1, pages - 2, 1]], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for row in table.tolist():
        for p in row:
            data[p] = torch.randn(2, 1, page, dim, generator=g, device=DEV)
    q = torch.randn(2, 16, dim, generator=g, device=DEV).to(torch.bfloat16)
    out, lse, ws = torch.empty_like(q), torch.empty(2, 16, device=DEV), plan.workspace()
    smq.sparse_mqa_attention_decode(plan, q, data[:, 0], data[:, 1], table, None,
                                    torch.tensor([180, 192], dtype=torch.int32, device=DEV), out, ws, lse=lse)
    assert smq.smq_get_status(ws) == 0
    for r, n in enumerate((180, 192)):
        both = data[table[r].long()].cpu().to(torch.float64).numpy()
        k, v = (both[:, side].transpose(0, 2, 1, 3).reshape(-1, 1, dim)[:n] for side in (0, 1))
        _check(out[r], lse[r], ref.attend(q[r].cpu().to(torch.float64).numpy(), k, v, dim ** -0.5), "bf16", f"row {r}")
    # the append writes there too
    kv = torch.randn(1, 1, dim, device=DEV).to(torch.bfloat16)
    smq.sparse_mqa_append_kv(plan, None, kv, kv, None, None, torch.tensor([(pages - 1) * page + 5], device=DEV), data[:, 0],
                             data[:, 1], ws)
    assert smq.smq_get_status(ws) == 0
    assert torch.equal(data[pages - 1, 0, 0, 5], kv[0, 0]) and torch.equal(data[pages - 1, 1, 0, 5], kv[0, 0])


def test_streams_and_graphs():
    """Calls on a stream of their own, and replayed from a graph on inputs that changed in place."""
    rng = np.random.Generator(np.random.PCG64(21))
    lens = [3000, 200, 77]
    cache = ref.Cache(rng, 1, 128, 64, "bf16", lens)
    rows = Rows(rng, cache, 16, [0, 1, 2])
    ke = torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV)
    call = smq.AttentionCall(rows.plan, rows.q_dev, row_ke=ke, **rows.dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    rows.check([np.arange(1)] * 3)
    with torch.cuda.graph(graph):
        call()
    ke.copy_(torch.tensor(lens, dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert smq.smq_get_status(rows.dev["workspace"]) == 0
    rows.check([np.arange(n) for n in lens])


def test_zero_rows_do_nothing():
    plan = smq.AttentionPlan(4, 2, 64, 16, max_rows=4)
    data = torch.zeros(2, 2, 2, 16, 64, device=DEV, dtype=torch.bfloat16)
    q = torch.empty(0, 4, 64, device=DEV, dtype=torch.bfloat16)
    ws = plan.workspace()
    smq.sparse_mqa_attention_decode(plan, q, data[:, 0], data[:, 1], torch.zeros(1, 1, dtype=torch.int32, device=DEV), None,
                                    torch.empty(0, dtype=torch.int32, device=DEV), torch.empty_like(q), ws)
    empty = torch.empty(0, 2, 64, device=DEV, dtype=torch.bfloat16)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    smq.sparse_mqa_append_kv(plan, None, empty, empty, None, None, none, data[:, 0], data[:, 1], ws)
    assert smq.smq_get_status(ws) == 0
