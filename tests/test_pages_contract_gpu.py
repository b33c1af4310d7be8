"""Tables and counts that do not agree before a call: what the page operators make of them does not depend on timing."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import pages_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAGE = 16


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Pool:
    """A pool on the GPU that calls begin from again and again."""

    def __init__(self, refs, table):
        self.table, self.refs = np.asarray(table, np.int32), np.asarray(refs, np.int32)
        self.plan = smq.PagePlan(PAGE, len(self.refs), *self.table.shape)
        self.ws = self.plan.workspace()

    def many(self, call, rounds=30):
        """The status, counts and table after a call, which have to be the same every time."""
        got = None
        for _ in range(rounds):
            refs, table = _i32(self.refs), _i32(self.table)
            call(self.plan, refs, table, self.ws)
            now = smq.smq_get_status(self.ws), refs.cpu().numpy(), table.cpu().numpy()
            got = got or now
            assert got[0] == now[0] and np.array_equal(got[1], now[1]) and np.array_equal(got[2], now[2])
        return got


@pytest.mark.parametrize("taker_first", [True, False])
def test_a_page_that_nobody_holds_is_taken_and_given_back(taker_first):
    """One row's table says that it holds the only free page, and gives it back; another takes that page."""
    columns, pages, nobody = 4096, 9000, 77
    taker, giver = (0, 1) if taker_first else (1, 0)
    for at in (0, columns - 1):
        refs = np.ones(pages)
        refs[nobody] = 0
        table = np.full((2, columns), -1)
        table[giver, at] = nobody
        end = [0, 0]
        end[taker] = PAGE
        b = Pool(refs, table)
        status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_resize(plan, r, t, _i32(end), ws))
        assert status == pages_ref.BOUNDS and after[taker, 0] == nobody and (after[giver] == -1).all()
        assert got[nobody] == 1, "the row that took it holds it"


@pytest.mark.parametrize("holders", [2, 3, 5])
def test_a_page_of_one_holder_that_several_rows_give_back(holders):
    columns = 300
    table = np.full((6, columns), -1)
    table[:holders, columns // 2] = 9
    refs = np.zeros(50)
    refs[9] = 1
    b = Pool(refs, table)
    status, got, _ = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_resize(plan, r, t, _i32([0] * 6), ws))
    assert status == pages_ref.BOUNDS and got[9] == 0
    # the same while forks share it: of its count and the additions, each give-back takes one
    status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_fork(
        plan, r, t, _i32([0, 5, 5, 5, 5][:holders]), _i32([5, 1, 2, 3, 4][:holders]),
        _i32([(columns // 2 + 1) * PAGE] + [0] * (holders - 1)), [], ws))
    assert after[5, columns // 2] == 9
    assert got[9] == max(0, 1 + 1 - (holders - 1))  # row 0 keeps its entry, the others give theirs back
    assert status == (pages_ref.BOUNDS if holders - 1 > 2 else 0)


def test_a_fork_takes_a_page_that_nobody_holds():
    """A fork's copy goes to the free page that another destination's table has."""
    columns, pages, nobody = 2000, 3000, 5
    refs = np.ones(pages)
    refs[nobody] = 0
    table = np.full((4, columns), -1)
    table[0, 0], table[1, columns - 1] = 8, nobody
    b = Pool(refs, table)
    for src, dst, n in (([0, 3], [2, 1], [5, 0]), ([3, 0], [1, 2], [0, 5])):
        status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_fork(plan, r, t, _i32(src), _i32(dst), _i32(n), [], ws))
        assert status == pages_ref.BOUNDS and after[2, 0] == nobody and got[nobody] == 1 and (after[1] == -1).all()


def test_counts_below_zero_stay():
    refs = np.array([-2, 1, 0, 0])
    b = Pool(refs, [[0, 1], [-1, -1]])
    status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_resize(plan, r, t, _i32([0, PAGE]), ws))
    assert status == pages_ref.BOUNDS and got.tolist() == [-2, 0, 1, 0] and after.tolist() == [[-1, -1], [2, -1]]
    status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_fork(
        plan, r, t, _i32([0]), _i32([1]), _i32([2 * PAGE]), [], ws))
    assert status == pages_ref.BOUNDS and got.tolist() == [-2, 2, 0, 0] and after.tolist() == [[0, 1], [-1, 1]]


@pytest.mark.parametrize("entry", [50, 2 ** 31 - 1])
def test_an_entry_past_the_pool_that_a_row_keeps(entry):
    """It is reported, as one that is given back is, and stays; the row's other columns have their pages."""
    refs = np.zeros(50)
    refs[[3, 4]] = 1
    b = Pool(refs, [[-1, entry, 3, -1], [4, -1, -1, entry]])
    status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_resize(plan, r, t, _i32([3 * PAGE, PAGE]), ws), 3)
    assert status == pages_ref.BOUNDS and after.tolist() == [[0, entry, 3, -1], [4, -1, -1, -1]]
    assert got.tolist() == [1, 0, 0, 1, 1] + [0] * 45
    status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_resize(
        plan, r, t, _i32([3 * PAGE]), ws, row_begin=_i32([PAGE])), 3)
    assert status == pages_ref.BOUNDS and after[0].tolist() == [-1, entry, 3, -1] and got.sum() == 2


def test_empty_ranges():
    """One that begins inside a page holds that page, one that begins at a page's start, or behind the end's page, holds none."""
    ranges = [(20, 20), (16, 16), (30, 17), (32, 20), (0, 0), (40, 33), (47, 48), (48, 48)]
    b = Pool(np.zeros(40), np.full((len(ranges), 5), -1))
    begin, end = zip(*ranges)
    status, got, after = b.many(lambda plan, r, t, ws: smq.sparse_mqa_pages_resize(plan, r, t, _i32(end), ws, row_begin=_i32(begin)), 3)
    held = [np.flatnonzero(row >= 0).tolist() for row in after]
    assert status == 0 and held == [[1], [], [1], [], [], [2], [2], []] and got.sum() == 4


def test_planes_that_share_bytes_are_not_compacted():
    """A token would move twice. Neighbours in a page, and whole pools behind one another, are taken."""
    plan = smq.PagePlan(PAGE, 6, 2, 3)
    refs, table = plan.state()
    ws = plan.workspace()
    smq.sparse_mqa_pages_resize(plan, refs, table, _i32([48, 48]), ws)
    start, keep = _i32([0, 3]), _i32([[5, 9, 40], [7, 20, -1]])
    data = torch.randint(0, 1 << 30, (12, 5, PAGE, 4), dtype=torch.int32, device=DEV)
    before = data.clone()
    a, b = data[:6], data[6:]
    for planes in ([a[:, :2], a[:, :2]], [a[:, :2], a[:, 1:3]], [a[:, 3:], b[:, :1], a[:, 4:]], [a, data[1:7]], [a, data[3:9, :1]],
                   [a, a[:, :1].view(torch.int16)]):
        with pytest.raises(smq.SMQError) as e:
            smq.sparse_mqa_cache_compact(plan, refs, table, start, keep, planes, ws)
        assert e.value.code == smq.SMQ_ERR_INVALID_ARG and torch.equal(data, before)
    smq.sparse_mqa_cache_compact(plan, refs, table, start, keep, [a[:, :2], a[:, 3:], b, a[:, 2:3]], ws)
    assert smq.smq_get_status(ws) == 0
    rows = table.cpu().numpy()
    want = before.clone()
    for pool in (0, 6):
        for r, (s, ids) in enumerate(((0, (5, 9, 40)), (3, (7, 20)))):
            for j, t in enumerate(ids):
                want[pool + rows[r, (s + j) // PAGE], :, (s + j) % PAGE] = before[pool + rows[r, t // PAGE], :, t % PAGE]
    assert torch.equal(data, want)
