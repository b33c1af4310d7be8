"""The page operators, through the public entry points, against a pool on the host: resize, fork and compact, alone, one after
another, and together with the attention that reads what they arrange."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import pages_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Both:
    """The same pool on the host and on the GPU, with planes of bf16 keys and values, scales and the indexer's pages."""

    def __init__(self, page_size, num_pages, rows, columns, kinds=("kv", "scales", "index"), seed=0, offset=0):
        self.host = pages_ref.Pool(page_size, num_pages, rows, columns)
        self.plan = smq.PagePlan(page_size, num_pages, rows, columns)
        store = torch.zeros(num_pages + offset, dtype=torch.int32, device=DEV)  # counts at any 4-byte address
        self.refs, self.table = store[offset:], self.plan.state()[1]
        self.ws = self.plan.workspace()
        g = torch.Generator(device=DEV).manual_seed(seed)

        def some(*shape):
            return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)

        self.planes, self.stores = [], []
        if "kv" in kinds:
            kv = some(num_pages, 2, 3, page_size, 128).view(torch.bfloat16)  # 3 kv heads of 64
            self.planes += [kv[:, 0], kv[:, 1]]
            self.stores.append(kv)
        if "scales" in kinds:
            sc = some(num_pages, 2, 3, page_size, 4).view(torch.int32).squeeze(-1)  # (bits: NaN would not compare)
            self.planes += [sc[:, 0], sc[:, 1]]
            self.stores.append(sc)
        if "index" in kinds:
            k = some(num_pages, page_size * 68)
            index = type("P", (), dict(page_bytes=68 * page_size, page_size=page_size, head_dim=128))
            self.planes += smq.indexer_planes(index, k)
            self.stores.append(k)
        if "odd" in kinds:  # 12 bytes a token, and a word between pages
            odd = some(num_pages, 5 * page_size * 12 + 4)
            self.planes.append(odd[:, :-4].unflatten(1, (5, page_size, 12)))
            self.stores.append(odd)
        self.host.planes = [self._bits(p) for p in self.planes]

    @staticmethod
    def _bits(t):
        return t.cpu().view(torch.int16).numpy().copy() if t.dtype == torch.bfloat16 else t.cpu().numpy().copy()

    def set(self, refs=None, table=None):
        if refs is not None:
            self.host.refs[:] = refs
        if table is not None:
            self.host.table[:] = table
        self.refs.copy_(torch.from_numpy(self.host.refs))
        self.table.copy_(torch.from_numpy(self.host.table))

    def same(self, got, want):
        status = smq.smq_get_status(self.ws)
        assert status == want, f"status {status}, expected {want}"
        assert np.array_equal(self.table.cpu().numpy(), self.host.table), "table"
        assert np.array_equal(self.refs.cpu().numpy(), self.host.refs), "counts"
        for i, (p, q) in enumerate(zip(self.planes, self.host.planes)):
            assert np.array_equal(self._bits(p), q), f"plane {i}"

    @staticmethod
    def _i32(x):
        return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)

    def resize(self, end, begin=None, keep_first=0, rows=None):
        want = self.host.resize(end, begin, keep_first, rows)
        self.same(smq.sparse_mqa_pages_resize(self.plan, self.refs, self.table, self._i32(end), self.ws, row_begin=self._i32(begin),
                                              keep_first=keep_first, rows=self._i32(rows)), want)
        return want

    def fork(self, src, dst, length):
        want = self.host.fork(src, dst, length)
        self.same(smq.sparse_mqa_pages_fork(self.plan, self.refs, self.table, self._i32(src), self._i32(dst), self._i32(length),
                                            self.planes, self.ws), want)
        return want

    def compact(self, start, keep, rows=None):
        want = self.host.compact(start, keep, rows)
        self.same(smq.sparse_mqa_cache_compact(self.plan, self.refs, self.table, self._i32(start), self._i32(keep), self.planes,
                                               self.ws, rows=self._i32(rows)), want)
        return want


def _rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def _pad(lists, width=None):
    width = width or max([len(x) for x in lists] + [1])
    return np.array([list(x) + [-1] * (width - len(x)) for x in lists], np.int32).reshape(len(lists), width)


# -------------------------------------------------------------------- resize


@pytest.mark.parametrize("page,pages,rows,columns", [(16, 100, 5, 7), (64, 3000, 40, 33), (1, 50, 3, 12), (5, 7, 1, 9),
                                                     (128, 4099, 130, 129)])
@pytest.mark.parametrize("offset", [0, 1])
def test_resize_matches(page, pages, rows, columns, offset):
    rng = _rng(page, pages)
    b = Both(page, pages, rows, columns, kinds=(), offset=offset)
    top = page * columns
    b.resize(rng.integers(0, top + 1, rows) // 2)
    b.resize(rng.integers(0, top + 1, rows), begin=rng.integers(-3, top + 1, rows))
    b.resize(rng.integers(0, top + 1, rows), begin=rng.integers(0, top + 1, rows), keep_first=page + 1)
    some = rng.permutation(rows)[: (rows + 1) // 2]
    b.resize(rng.integers(-5, top // 3 + 1, len(some)), rows=some)
    b.resize(np.zeros(rows))
    assert not b.host.refs.any() and (b.host.table == -1).all()


def test_resize_of_a_large_pool():
    """A pool past one cluster's first pass, free pages far apart, a table wider than a warp's step."""
    rng = _rng(3)
    pages, rows, columns = 300007, 300, 700
    b = Both(8, pages, rows, columns, kinds=())
    b.set(refs=(rng.random(pages) < 0.3) * rng.integers(1, 4, pages))
    b.resize(rng.integers(0, 8 * columns, rows))
    end = rng.integers(0, 8 * columns, rows)
    b.resize(end, begin=end - 2000, keep_first=9)


def test_pages_run_out():
    b = Both(16, 10, 4, 8, kinds=())
    assert b.resize([80, 64, 50, 10]) == pages_ref.NO_PAGES
    assert b.resize([0, 64, 0, 0]) == 0
    assert b.resize([30, 64, 0, 128]) == pages_ref.NO_PAGES


def test_resize_reports_what_does_not_fit():
    b = Both(16, 40, 4, 8, kinds=())
    assert b.resize([100, 20, 30, 40]) == 0
    assert b.resize([50, 129, 16], rows=[0, 1, 2]) == pages_ref.BOUNDS           # past the table's row: cut there
    assert b.resize([1, 2, 3, 4], rows=[3, -1, 4, 3]) == pages_ref.BOUNDS        # no such rows, and one listed twice
    assert b.resize([20, 20], begin=[2 ** 31 - 1, -2 ** 31], rows=[0, 1]) == pages_ref.BOUNDS
    table = b.host.table.copy()
    table[2, 0] = 40                                                              # no such page
    b.set(table=table)
    assert b.resize([0], rows=[2]) == pages_ref.BOUNDS
    table = b.host.table.copy()
    free = int(np.flatnonzero(b.host.refs == 0)[-1])
    table[3, 7] = free                                                            # a page that nobody holds
    b.set(table=table)
    assert b.resize([0], rows=[3]) == pages_ref.BOUNDS
    assert (b.host.refs >= 0).all()


# ---------------------------------------------------------------------- fork


@pytest.mark.parametrize("kinds", [("kv",), ("kv", "scales", "index"), ("odd",), ()])
@pytest.mark.parametrize("page", [16, 5, 1])
def test_fork_matches(page, kinds):
    rng = _rng(page, len(kinds))
    rows, columns = 12, 9
    b = Both(page, 160, rows, columns, kinds=kinds)
    lens = rng.integers(0, page * columns + 1, rows)
    lens[0] = page * columns
    b.resize(lens)
    b.fork([0, 0, 0], [9, 10, 11], [page * 3, page * 3 + page // 2, page * columns])
    # beams: every row from a random one, some from themselves
    src = rng.integers(0, rows, rows)
    length = lens[src] - rng.integers(0, 3, rows)
    b.fork(src, rng.permutation(rows), length)
    b.fork(rng.permutation(rows), np.arange(rows), lens)
    b.fork([3, 4], [4, 3], [lens[3], lens[4]])  # two rows change places
    b.resize(np.zeros(rows))
    assert not b.host.refs.any()


def test_fork_of_a_row_with_a_window():
    """Columns that a window has given back are not there in the fork either, not even the one that it would copy."""
    b = Both(16, 60, 4, 10)
    b.resize([150], begin=[70], keep_first=4, rows=[0])
    b.fork([0, 0, 0], [1, 2, 3], [150, 5, 40])


def test_many_forks_of_one_prompt():
    b = Both(64, 1500, 400, 21, kinds=("kv",))
    b.resize([1300], rows=[7])
    dst = [r for r in range(400) if r != 7]
    b.fork([7] * 399, dst, [1300 - i for i in range(399)])


def test_forks_without_pages_left():
    b = Both(16, 8, 5, 4)
    b.resize([40], rows=[0])
    assert b.fork([0] * 4, [1, 2, 3, 4], [40, 20, 32, 39]) == 0
    assert b.fork([0] * 4, [1, 2, 3, 4], [33, 34, 35, 36]) == pages_ref.NO_PAGES


def test_fork_reports_what_does_not_fit():
    b = Both(16, 60, 6, 6)
    b.resize([90, 90, 20, 0, 0, 0])
    assert b.fork([0, 7, 1, -1], [3, 4, 3, 5], [50, 50, 50, 50]) == pages_ref.BOUNDS  # no such sources, 3 listed twice
    assert b.fork([0, 1], [6, 5], [50, 97]) == pages_ref.BOUNDS                        # no such row; longer than a row
    assert b.fork([0], [4], [-4]) == 0
    table = b.host.table.copy()
    table[1, 1], table[1, 2] = 60, int(np.flatnonzero(b.host.refs == 0)[0])            # no such page; nobody's page
    b.set(table=table)
    assert b.fork([1], [4], [90]) == pages_ref.BOUNDS


# ------------------------------------------------------------------- compact


@pytest.mark.parametrize("kinds", [("kv",), ("kv", "scales", "index"), ("odd",)])
@pytest.mark.parametrize("page,columns", [(16, 40), (7, 60), (64, 9), (1, 200)])
def test_compact_matches(page, columns, kinds):
    rng = _rng(page, columns)
    rows = 9
    b = Both(page, rows * columns + 3, rows, columns, kinds=kinds)
    top = page * columns
    b.resize(np.full(rows, top))
    for density in (0.02, 0.5, 0.97, 1.0):
        start = rng.integers(0, top // 2, rows)
        keep = [np.flatnonzero(rng.random(top - s) < density) + s for s in start]
        b.compact(start, _pad(keep))
    some = rng.permutation(rows)[:3]
    b.compact([0, 1, top - 1], _pad([[top - 1], [], [top - 1]]), rows=some)
    b.compact([0, 5, 2], _pad([np.arange(top - 5), np.arange(5, top), np.arange(top // 2, top)], top), rows=some)


def test_compact_of_a_long_row():
    """Longer than every block checks for itself, many chunks whose places are sources of others."""
    rng = _rng(5)
    page, columns = 32, 300
    b = Both(page, 2 * columns, 2, columns, kinds=("kv", "scales"))
    b.resize([page * columns] * 2)
    b.compact([4, 0], _pad([np.flatnonzero(rng.random(page * columns - 4) < 0.9) + 4, [3]]))
    b.compact([1, 0], _pad([np.arange(2, page * columns), np.arange(1, page * columns)]))


@pytest.mark.parametrize("width", [2048, 2044, 1040, 4])
def test_tokens_of_every_size(width):
    """The longest tokens of a plane, in pieces of 16 bytes and of 4, and the shortest."""
    rng = _rng(width)
    b = Both(8, 70, 4, 12, kinds=())
    store = torch.randint(0, 256, (70, 2, 8, width), device=DEV, dtype=torch.uint8)
    b.planes, b.stores = [store], [store]
    b.host.planes = [b._bits(store)]
    b.resize([90, 96, 50, 0])
    b.compact([3, 0, 10], _pad([np.flatnonzero(rng.random(87) < 0.7) + 3, np.arange(48, 96), np.arange(10, 50)]), rows=[0, 1, 2])
    long = np.full((1, 1100), -1, np.int32)
    long[0, :60] = np.sort(rng.permutation(90)[:60])
    b.compact([0], long, rows=[0])
    b.fork([0, 1], [3, 2], [61, 95])


def test_compact_refuses_rows_whole():
    b = Both(16, 40, 6, 5)
    b.resize([80, 80, 80, 80, 80, 40])
    good = [3, 9, 20, 40]
    for start, ids in (([0] * 6, [good, [3, 3], [5, 4], [3, 80], good, [3, 50]]),   # not ascending, past the table, no page
                       ([4, -1, 0, 10, 3, 0], [good, good, [0, 1, 1], [9], good, []]),  # before the start
                       ([79, 0, 2 ** 31 - 1, 0, 0, 0], [[79], [79], [5], [2 ** 31 - 1], [], []])):
        assert b.compact(start, _pad(ids)) == pages_ref.BOUNDS
    assert b.compact([0, 0, 0], _pad([good] * 3), rows=[2, 2, 6]) == pages_ref.BOUNDS
    # a place that two rows hold
    b.resize([0], rows=[5])
    b.fork([0], [5], [80])
    assert b.compact([0, 0], _pad([good, good]), rows=[0, 1]) == pages_ref.BOUNDS
    assert b.compact([0, 0], _pad([[0, 1, 2], good]), rows=[0, 1]) == 0             # nothing moves
    long = np.full((2, 1500), -1, np.int32)                                         # the same through the check of long lists
    long[:, :4] = good
    assert b.compact([0, 0], long, rows=[0, 1]) == pages_ref.BOUNDS
    table = b.host.table.copy()
    table[2, 1] = 40
    b.set(table=table)
    assert b.compact([0], _pad([[3, 20]]), rows=[2]) == pages_ref.BOUNDS


def test_shared_pages_are_read():
    """Kept tokens may come from pages that others hold, as long as the places are the row's own."""
    b = Both(16, 60, 3, 8)
    b.resize([100], rows=[0])
    b.fork([0], [1], [64 + 30])   # rows 0 and 1 share five whole pages
    b.resize([110], rows=[1])
    assert b.compact([80], _pad([[81, 90, 93]]), rows=[1]) == 0
    assert b.compact([30], _pad([[81]]), rows=[1]) == pages_ref.BOUNDS


# ------------------------------------------------------------------ together


def test_a_pool_through_many_steps():
    rng = _rng(11)
    page, rows, columns = 16, 10, 12
    b = Both(page, 90, rows, columns)
    lens = np.zeros(rows, int)
    for step in range(40):
        what = rng.integers(0, 3)
        if what == 0:
            lens = np.maximum(0, np.minimum(page * columns, lens + rng.integers(-60, 90, rows)))
            b.resize(lens)
        elif what == 1:
            n = int(rng.integers(1, rows + 1))
            src, dst = rng.integers(0, rows, n), rng.permutation(rows)[:n]
            length = lens[src]
            b.fork(src, dst, length)
            lens[dst] = np.where(src == dst, lens[dst], length)
        else:
            start, keep = [], []
            for r in range(rows):
                s = int(rng.integers(0, lens[r] + 1))
                start.append(s)
                keep.append(np.flatnonzero(rng.random(lens[r] - s) < 0.6) + s)
            b.compact(start, _pad(keep))
    b.resize(np.zeros(rows))
    assert not b.host.refs.any()


def test_streams_and_graphs():
    """Replayed from a graph on lengths that change in place; two pools at once on two streams."""
    pools = [Both(16, 200, 8, 10, seed=i) for i in range(2)]
    end = [torch.tensor([30 + i] * 8, dtype=torch.int32, device=DEV) for i in range(2)]
    calls = [smq.ResizeCall(b.plan, b.refs, b.table, e, b.ws) for b, e in zip(pools, end)]
    torch.cuda.synchronize()
    for call in calls:
        with torch.cuda.stream(torch.cuda.Stream()):
            call()
    torch.cuda.synchronize()
    for i, b in enumerate(pools):
        b.same(None, b.host.resize([30 + i] * 8))
    b = pools[0]
    src, dst, n = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1, 2], [4, 5, 6], [30, 20, 16]))
    start, keep = torch.tensor([17] * 8, dtype=torch.int32, device=DEV), torch.tensor([[20, 25, 29]] * 8, dtype=torch.int32, device=DEV)
    fork = smq.ForkCall(b.plan, b.refs, b.table, src, dst, n, b.planes, b.ws)
    compact = smq.CompactCall(b.plan, b.refs, b.table, start, keep, b.planes, b.ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls[0]()
        compact()
        fork()
    for length in (30, 100, 64, 31):
        end[0].fill_(length)
        graph.replay()
        torch.cuda.synchronize()
        want = b.host.resize([length] * 8)
        want |= b.host.compact([17] * 8, np.array([[20, 25, 29]] * 8))
        b.same(None, want | b.host.fork([0, 1, 2], [4, 5, 6], [30, 20, 16]))


def test_no_rows():
    b = Both(16, 20, 3, 4)
    none = np.zeros(0, np.int32)
    b.resize(none)
    b.fork(none, none, none)
    b.compact(none, np.zeros((0, 2), np.int32))


# ------------------------------------------------------------------ refusals

BAD = smq.SMQ_ERR_INVALID_ARG


def _calls():
    b = Both(16, 20, 4, 4)
    x = torch.zeros(3, dtype=torch.int32, device=DEV)
    y = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)
    return b, {"resize": smq.ResizeCall(b.plan, b.refs, b.table, x, b.ws, row_begin=x, rows=y),
               "fork": smq.ForkCall(b.plan, b.refs, b.table, x, y, x, b.planes, b.ws),
               "compact": smq.CompactCall(b.plan, b.refs, b.table, x, torch.full((3, 2), -1, dtype=torch.int32, device=DEV),
                                          b.planes, b.ws, rows=y)}


@pytest.mark.parametrize("op,field,value,code", [
    (op, f, v, c) for op in ("resize", "fork", "compact") for f, v, c in (
        ("num_rows", -1, BAD), ("num_rows", 5, BAD), ("block_table", None, BAD), ("page_refs", None, BAD),
        ("workspace", None, BAD), ("workspace_bytes", 256, smq.SMQ_ERR_WORKSPACE_TOO_SMALL), ("struct_size", 8, BAD))
] + [
    ("resize", "row_end", None, BAD), ("resize", "keep_first", -1, BAD), ("resize", "rows", 2, BAD),
    ("fork", "src_rows", None, BAD), ("fork", "dst_rows", None, BAD), ("fork", "row_len", None, BAD),
    ("fork", "num_planes", 9, BAD), ("fork", "num_planes", -1, BAD), ("fork", "planes", None, BAD),
    ("compact", "row_start", None, BAD), ("compact", "keep_ids", None, BAD), ("compact", "num_keep", 0, BAD),
    ("compact", "num_keep", 3, BAD), ("compact", "keep_ld", 1, BAD), ("compact", "num_planes", 0, BAD),
    ("compact", "num_planes", 9, BAD),
])
def test_the_library_refuses_bad_arguments(op, field, value, code):
    b, calls = _calls()
    setattr(calls[op].args, field, value)
    with pytest.raises(smq.SMQError) as e:
        calls[op]()
    assert e.value.code == code
    b.same(None, 0)


@pytest.mark.parametrize("field,value,code", [
    ("base", None, BAD), ("base", 2, BAD), ("page_stride", 6, BAD), ("page_stride", 4, BAD), ("vectors", 0, BAD), ("token_bytes", 0, BAD),
    ("token_bytes", 6, BAD), ("vectors", 1025, smq.SMQ_ERR_UNSUPPORTED), ("token_bytes", 2052, smq.SMQ_ERR_UNSUPPORTED),
])
def test_the_library_refuses_bad_planes(field, value, code):
    for op in ("fork", "compact"):
        b, calls = _calls()
        setattr(calls[op].args.planes[1], field, value)
        with pytest.raises(smq.SMQError) as e:
            calls[op]()
        assert e.value.code == code
        b.same(None, 0)


def test_the_binding_refuses_what_does_not_fit():
    b, _ = _calls()
    x = torch.zeros(3, dtype=torch.int32, device=DEV)
    keep = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    for error, make in (
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs, b.table, x.cpu(), b.ws)),
            (TypeError, lambda: smq.ResizeCall(b.plan, b.refs, b.table, x.long(), b.ws)),
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs, b.table, x, b.ws, rows=x[:2])),
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs, b.table, x, b.ws, row_begin=x[:2])),
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs, b.table, torch.zeros(5, dtype=torch.int32, device=DEV), b.ws)),
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs[:3], b.table, x, b.ws)),
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs, b.table[:, :3], x, b.ws)),
            (ValueError, lambda: smq.ResizeCall(b.plan, b.refs, b.table[:3], x, b.ws)),
            (ValueError, lambda: smq.ForkCall(b.plan, b.refs, b.table, x, x[:2], x, b.planes, b.ws)),
            (ValueError, lambda: smq.ForkCall(b.plan, b.refs, b.table, x, x, x, [b.planes[0][:3]], b.ws)),
            (ValueError, lambda: smq.ForkCall(b.plan, b.refs, b.table, x, x, x, [b.planes[0].transpose(1, 3)], b.ws)),
            (ValueError, lambda: smq.ForkCall(b.plan, b.refs, b.table, x, x, x, b.planes * 2, b.ws)),
            (ValueError, lambda: smq.ForkCall(b.plan, b.refs, b.table, x, x, x, [b.planes[0].cpu()], b.ws)),
            (ValueError, lambda: smq.ForkCall(b.plan, b.refs, b.table, x, x, x, [torch.zeros(20, 1, 16, dtype=torch.uint8, device=DEV)], b.ws)),
            (ValueError, lambda: smq.CompactCall(b.plan, b.refs, b.table, x, keep[:2], b.planes, b.ws)),
            (ValueError, lambda: smq.CompactCall(b.plan, b.refs, b.table, x, keep.t(), b.planes, b.ws)),
            (ValueError, lambda: smq.indexer_planes(type("P", (), dict(page_bytes=5, page_size=16, head_dim=128)), b.stores[-1]))):
        with pytest.raises(error):
            make()


@pytest.mark.parametrize("bad,code", [
    (dict(page_size=0), BAD), (dict(page_size=65537), smq.SMQ_ERR_UNSUPPORTED), (dict(num_pages=0), BAD),
    (dict(num_pages=2 ** 31), smq.SMQ_ERR_UNSUPPORTED), (dict(table_rows=0), BAD), (dict(table_rows=8193), smq.SMQ_ERR_UNSUPPORTED),
    (dict(table_columns=0), BAD), (dict(table_columns=2 ** 20 + 1), smq.SMQ_ERR_UNSUPPORTED),
    (dict(table_rows=8192, table_columns=2 ** 20), smq.SMQ_ERR_UNSUPPORTED), (dict(device=99), smq.SMQ_ERR_CUDA),
])
def test_plans_that_are_refused(bad, code):
    with pytest.raises(smq.SMQError) as e:
        smq.PagePlan(**{**dict(page_size=16, num_pages=10, table_rows=4, table_columns=4), **bad})
    assert e.value.code == code
