"""Steps of drafted decoding over a paged cache, from the pages to the accepted tokens.

    python examples/draft_tree_step.py

A batch of sequences shares a pool of pages; two of them are samples of one prompt. In each step every sequence has a small
tree of drafted tokens behind its context:
  1. sparse_mqa_pages_resize takes pages for the trees;
  2. sparse_mqa_append_kv rotates the drafted queries and keys and writes keys and values into the pages;
  3. sparse_mqa_attention_tree attends from each drafted token to the context and to its ancestors, and, as a sliding layer
     would, sparse_mqa_attention_window from the first token of each tree;
  4. sparse_mqa_cache_compact moves the accepted path of each tree to the front of it;
  5. sparse_mqa_pages_resize gives back the pages behind.
At the start sparse_mqa_pages_fork makes the second sample of the prompt.
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_top_expand_gb300 as smq

HEADS, KV_HEADS, DIM, PAGE = 64, 8, 128, 64
NODES, WINDOW, SINKS = 12, 512, 4
LONGEST = 8192


class Batch:
    """The buffers that a serving loop keeps, for contexts of the given lengths and a second sample of the first of them."""

    def __init__(self, lens, cache_dtype="bf16", seed=0):
        dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.generator = dev, torch.Generator(device=dev).manual_seed(seed)
        rows, columns = len(lens) + 1, LONGEST // PAGE
        pages = sum(-(-(n + 64 * NODES) // PAGE) for n in lens) + 2 * rows + columns
        self.pool = smq.PagePlan(PAGE, pages, rows, columns)
        self.refs, self.table = self.pool.state()
        self.plan = smq.AttentionPlan(HEADS, KV_HEADS, DIM, PAGE, max_rows=4096, cache_dtype=cache_dtype)
        kind = torch.bfloat16 if cache_dtype == "bf16" else torch.uint8
        self.kv = torch.zeros(pages, 2, KV_HEADS, PAGE, DIM, device=dev, dtype=kind)
        self.scales = torch.ones(pages, 2, KV_HEADS, PAGE, device=dev) if cache_dtype == "e4m3" else None
        half = DIM // 2
        angle = torch.arange(LONGEST, device=dev).float().unsqueeze(1) * torch.exp(
            torch.arange(half, device=dev).float() * (-math.log(10000.0) / half))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        self.ws = self.plan.workspace(), self.plan.sequence_workspace(), self.pool.workspace()
        self.lens = torch.tensor(lens + [0], device=dev)
        self._resize(self.lens)
        for r, n in enumerate(lens):  # the contexts, through the same calls
            at = torch.arange(n, device=dev)
            for chunk in at.split(4096):
                self._append(torch.full_like(chunk, r), chunk, None)
        one = lambda x: torch.tensor([x], device=dev, dtype=torch.int32)  # noqa: E731
        smq.sparse_mqa_pages_fork(self.pool, self.refs, self.table, one(0), one(len(lens)), one(lens[0]), self._planes(), self.ws[2])
        self.lens[len(lens)] = lens[0]

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.generator, device=self.device, dtype=torch.bfloat16)

    def sides(self):
        s = self.scales
        return dict(k_cache=self.kv[:, 0], v_cache=self.kv[:, 1], k_scales=None if s is None else s[:, 0],
                    v_scales=None if s is None else s[:, 1])

    def _planes(self):
        return [x for x in self.sides().values() if x is not None]

    def _resize(self, lens):
        smq.sparse_mqa_pages_resize(self.pool, self.refs, self.table, lens.int(), self.ws[2])

    def _append(self, rows, at, q, positions=None):
        """Keys and values (random ones here) of positions `at` of rows, and queries turned by `positions`."""
        slots = self.table[rows, at // PAGE].long() * PAGE + at % PAGE
        out = None if q is None else torch.empty_like(q)
        smq.sparse_mqa_append_kv(self.plan, q, self.randn(len(at), KV_HEADS, DIM), self.randn(len(at), KV_HEADS, DIM),
                                 at if positions is None else positions, self.cos_sin, slots, workspace=self.ws[0], q_out=out,
                                 **self.sides())
        return out

    def draft(self):
        """A tree for every sequence: parents, ancestors as bits (the node itself among them), depths."""
        rows = len(self.lens)
        parent = (torch.rand(rows, NODES, generator=self.generator, device=self.device) *
                  torch.arange(NODES, device=self.device)).long()
        bits, depth = torch.zeros(rows, NODES, dtype=torch.int64, device=self.device), torch.zeros_like(parent)
        every = torch.arange(rows, device=self.device)
        for j in range(NODES):
            if j:
                bits[:, j] = bits[every, parent[:, j]]
                depth[:, j] = depth[every, parent[:, j]] + 1
            bits[:, j] |= 1 << j
        return bits, depth

    def step(self):
        """One step: the tree attention's results [rows, NODES, H, D], the window's of the first nodes, accepted tokens."""
        rows, dev = len(self.lens), self.device
        bits, depth = self.draft()
        self._resize(self.lens + NODES)
        row = torch.arange(rows, device=dev).repeat_interleave(NODES)
        at = (self.lens.unsqueeze(1) + torch.arange(NODES, device=dev)).flatten()
        q = self._append(row, at, self.randn(rows * NODES, HEADS, DIM), (self.lens.unsqueeze(1) + depth).flatten())
        out = torch.empty_like(q)
        cu = torch.arange(rows + 1, device=dev, dtype=torch.int32)
        smq.sparse_mqa_attention_tree(self.plan, q, block_table=self.table, cu_rows=cu * NODES, seq_len=(self.lens + NODES).int(),
                                      max_seq_rows=NODES, out=out, workspace=self.ws[1], tree_mask=bits.int().view(-1, 1),
                                      **self.sides())
        first = q.view(rows, NODES, HEADS, DIM)[:, 0].contiguous()
        local = torch.empty_like(first)
        smq.sparse_mqa_attention_window(self.plan, first, block_table=self.table, cu_rows=cu, seq_len=(self.lens + 1).int(),
                                        max_seq_rows=1, out=local, workspace=self.ws[1], window=WINDOW, sinks=SINKS, **self.sides())
        # what a verification accepts: here the path to the last node
        path = (bits[:, -1:] >> torch.arange(NODES, device=dev)) & 1
        ids = torch.where(path == 1, self.lens.unsqueeze(1) + torch.arange(NODES, device=dev), 1 << 30).sort(1).values
        keep = torch.where(ids < 1 << 30, ids, -1).int()
        smq.sparse_mqa_cache_compact(self.pool, self.refs, self.table, self.lens.int(), keep, self._planes(), self.ws[2])
        accepted = path.sum(1)
        self.lens = self.lens + accepted
        self._resize(self.lens)
        for ws in self.ws:
            if smq.smq_get_status(ws):
                raise RuntimeError("a call reported an error")
        return out.view(rows, NODES, HEADS, DIM), local, accepted


def main():
    batch = Batch([1500, 300, 64, 4000])
    for n in range(4):
        _, _, accepted = batch.step()
        print(f"step {n}: accepted", accepted.tolist(), "contexts", batch.lens.tolist(), "pages held", int((batch.refs > 0).sum()))


if __name__ == "__main__":
    main()
