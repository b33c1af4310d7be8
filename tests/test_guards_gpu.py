"""What the sequences' attention and the page operators write: their outputs and their workspace, of the sizes that they say, and
nothing beside them. Buffers lie between guard words, integer inputs and the cache are compared after the calls."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import sequence_ref as ref
from test_pages_gpu import Both

pytestmark = pytest.mark.gpu

DEV = "cuda"
GUARD = 1 << 16  # bytes on either side


def _rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


class Guarded:
    """Tensors between guard bytes."""

    def __init__(self):
        self.stores = []

    def __call__(self, shape, dtype):
        size = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        store = torch.full((2 * GUARD + size,), 0xA5, dtype=torch.uint8, device=DEV)
        self.stores.append((store, size))
        return store[GUARD:GUARD + size].view(dtype).view(shape)

    def check(self):
        for store, size in self.stores:
            assert (store[:GUARD] == 0xA5).all() and (store[GUARD + size:] == 0xA5).all(), f"written beside a buffer of {size} bytes"


GEOMETRIES = [  # heads, kv heads, dim, page, dtype: groups of 3, 24, 33, 41, 8, 128 and 1
    (6, 2, 128, 16, "bf16"), (24, 1, 64, 32, "bf16"), (33, 1, 128, 5, "bf16"), (41, 1, 64, 24, "e4m3"), (64, 8, 128, 64, "bf16"),
    (64, 8, 128, 64, "e4m3"), (128, 1, 64, 64, "bf16"), (3, 3, 128, 64, "e4m3"),
]
BATCHES = [
    [(1, 9000)],                                                        # one item over every CTA
    [(3, 300), (1, 1), (0, 9), (4, 1000)],                              # a tile of queries and less, items cut in two
    [(150, 700), (2, 40), (300, 300), (7, 7)],                          # two tiles of queries
    [(1 + i % 3, 5 + 13 * i % 400) for i in range(100)],                # more sequences than a warp's lanes
]


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", GEOMETRIES)
@pytest.mark.parametrize("seqs", BATCHES, ids=["long", "short", "many-rows", "many"])
@pytest.mark.parametrize("tree", [False, True])
def test_the_sequences_attention_writes_its_buffers_only(heads, kv_heads, dim, page, dtype, seqs, tree):
    rng = _rng(heads, dim, len(seqs))
    b = ref.Batch(rng, heads, kv_heads, dim, page, dtype, seqs, pad=5)
    g = Guarded()
    out, lse = g((b.rows, heads, dim), torch.bfloat16), g((b.rows, heads), torch.float32)
    ws = g((b.plan.sequence_workspace_size(),), torch.uint8)
    smq.smq_attn_workspace_init(b.plan, ws)
    inputs = [b.q, torch.from_numpy(b.table), torch.from_numpy(b.cu), torch.tensor([x for _, x in seqs], dtype=torch.int32),
              torch.from_numpy(b.order), b.cache.data] + ([] if b.cache.scales is None else [b.cache.scales])
    longest = max(n for n, _ in seqs)
    if tree:
        masks = [m for n, _ in seqs for m in ref.random_tree(rng, n)]
        inputs.append(torch.from_numpy(ref.pack(masks + [set(range(32))] * 5, max(1, -(-longest // 32)))))
    own = []
    for x in inputs:
        own.append(g(x.shape, x.dtype))
        own[-1].copy_(x)
    q, table, cu, lens, order, data = own[:6]
    scales = None if b.cache.scales is None else own[6]
    out.fill_(9)
    lse.fill_(9)
    what = dict(tree_mask=own[-1]) if tree else dict(window=200, sinks=3)
    call = smq.SequenceAttentionCall(b.plan, q, data[:, 0], data[:, 1], table, cu, lens, longest, out, ws, seq_indices=order, lse=lse,
                                     k_scales=None if scales is None else scales[:, 0],
                                     v_scales=None if scales is None else scales[:, 1], **what)
    for _ in range(3):
        call()
    assert smq.smq_get_status(ws) == 0
    g.check()
    for x, y in zip(inputs, own):
        assert torch.equal(x.to(DEV).view(torch.uint8), y.view(torch.uint8)), "an input"
    assert (out[int(b.cu[-1]):] == 9).all() and (lse[int(b.cu[-1]):] == 9).all()
    if not tree:  # rows among them, against the plain form
        b.out, b.lse = out, lse
        b.check([ref.window_sets(n, length, 200, 3) for n, length in seqs], rows={0, 1, longest // 2, longest - 1})


@pytest.mark.parametrize("page,pages,rows,columns", [(16, 100, 5, 7), (5, 4099, 40, 33), (64, 12289, 130, 65), (1, 50, 3, 12)])
def test_the_page_operators_write_their_buffers_only(page, pages, rows, columns):
    rng = _rng(page, pages)
    b = Both(page, pages, rows, columns, kinds=("scales",) if pages > 1000 else ("kv", "scales", "odd"))
    g = Guarded()
    refs, table = g((pages,), torch.int32), g((rows, columns), torch.int32)
    refs.copy_(b.refs)
    table.copy_(b.table)
    b.refs, b.table, b.ws = refs, table, g((b.plan.workspace_size(),), torch.uint8)
    smq.smq_page_workspace_init(b.plan, b.ws)
    top = page * columns
    for _ in range(3):
        lens = rng.integers(0, min(top, pages * page // rows // 2) + 1, rows)
        b.resize(lens)
        src = rng.integers(0, rows, rows)
        b.fork(src, rng.permutation(rows), np.maximum(0, lens[src] - rng.integers(0, 3, rows)))
        b.resize(np.minimum(top, lens + page), begin=lens // 2, keep_first=page // 2)
        b.resize(np.zeros(rows))
        b.resize(lens)
        start = rng.integers(0, lens // 2 + 1)
        keep = np.full((rows, max(1, int(lens.max()))), -1, np.int32)
        for i in range(rows):
            ids = np.flatnonzero(rng.random(lens[i] - start[i]) < 0.6) + start[i]
            keep[i, :len(ids)] = ids
        b.compact(start, keep)
        b.compact(start, np.pad(keep, ((0, 0), (0, 1100)), constant_values=-1))
        g.check()
