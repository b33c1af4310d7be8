"""One decode step of two-level sparse attention, from a step's projections to its attention output.

    python examples/sparse_decode_step.py

For a batch of sequences with cached contexts, each with one new token:
  1. sparse_mqa_append_kv rotates the new queries and keys and appends keys and values to the attention cache;
  2. sparse_mqa_write_k_cache and sparse_mqa_quantize_q make the indexer's key and queries;
  3. sparse_mqa_candidate_source_decode publishes each row's candidate blocks (the source layer's part), and
     sparse_mqa_logits_topk_decode selects the top-k tokens inside them;
  4. sparse_mqa_attention_selected attends over the selected tokens.
sparse_mqa_attention_decode over the whole context stands beside it: where the selection covers the context, both agree.
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_top_expand_gb300 as smq

HEADS, KV_HEADS, DIM, PAGE = 64, 1, 128, 64        # attention
INDEX_HEADS, BLOCK, BLOCKS, TOPK = 64, 128, 32, 2048  # indexer
CHUNK = 4096  # tokens of a prefill call


class Step:
    """The buffers that a serving loop keeps, for `rows` sequences of up to `longest` tokens."""

    def __init__(self, lens, longest, cache_dtype="bf16", seed=0):
        dev = torch.device("cuda", torch.cuda.current_device())
        g = torch.Generator(device=dev).manual_seed(seed)
        rows = len(lens)
        self.attn = smq.AttentionPlan(HEADS, KV_HEADS, DIM, PAGE, max_rows=max(rows, CHUNK), cache_dtype=cache_dtype)
        self.index = smq.Plan(INDEX_HEADS, PAGE, BLOCK, BLOCKS, TOPK, max_rows=rows)
        width = -(-longest // PAGE)
        pages = rows * width
        self.table = torch.randperm(pages, generator=g, device=dev).int().view(rows, width).contiguous()
        kind = torch.bfloat16 if cache_dtype == "bf16" else torch.uint8
        self.kv = torch.zeros(pages, 2, KV_HEADS, PAGE, DIM, device=dev, dtype=kind)
        self.scales = torch.ones(pages, 2, KV_HEADS, PAGE, device=dev) if cache_dtype == "e4m3" else None
        self.k_index = torch.zeros(pages, self.index.page_bytes, device=dev, dtype=torch.uint8)
        half = DIM // 2
        angle = torch.arange(longest, device=dev).float().unsqueeze(1) * torch.exp(
            torch.arange(half, device=dev).float() * (-math.log(10000.0) / half))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        self.ws_attn, self.ws_index = self.attn.workspace(), self.index.workspace(rows)
        self.longest = longest
        self.ws_source = torch.empty(smq.smq_source_workspace_size(self.index, rows, longest), device=dev, dtype=torch.uint8)
        smq.smq_workspace_init(self.index, self.ws_source)
        self.lens = torch.tensor(lens, device=dev, dtype=torch.int64)  # tokens before this step
        self.generator, self.device = g, dev
        self._prefill()

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.generator, device=self.device, dtype=torch.bfloat16)

    def sides(self):
        s = self.scales
        return dict(k_cache=self.kv[:, 0], v_cache=self.kv[:, 1], k_scales=None if s is None else s[:, 0],
                    v_scales=None if s is None else s[:, 1])

    def slots(self, rows, positions):
        return self.table[rows, positions // PAGE].long() * PAGE + positions % PAGE

    def _prefill(self):
        """Fill the contexts with random keys and values, through the same calls."""
        for r, n in enumerate(self.lens.tolist()):
            for start in range(0, n, CHUNK):
                at = torch.arange(start, min(n, start + CHUNK), device=self.device)
                slots = self.slots(torch.full_like(at, r), at)
                k, v = self.randn(len(at), KV_HEADS, DIM), self.randn(len(at), KV_HEADS, DIM)
                smq.sparse_mqa_append_kv(self.attn, None, k, v, at, self.cos_sin, slots, workspace=self.ws_attn, **self.sides())
                smq.sparse_mqa_write_k_cache(self.index, self.randn(len(at), DIM), slots, self.k_index, self.ws_index)

    def run(self):
        """One token for every sequence: its attention output [rows, H, D] over the selected tokens, the same over the
        whole context, and the selected ids."""
        rows, dev = len(self.lens), self.device
        width = (HEADS + 2 * KV_HEADS) * DIM
        qkv = self.randn(rows, width)  # the fused projection of the step
        q = qkv[:, :HEADS * DIM].view(rows, HEADS, DIM)
        k = qkv[:, HEADS * DIM:-KV_HEADS * DIM].view(rows, KV_HEADS, DIM)
        v = qkv[:, -KV_HEADS * DIM:].view(rows, KV_HEADS, DIM)
        slots = self.slots(torch.arange(rows, device=dev), self.lens)
        q_rot = torch.empty(rows, HEADS, DIM, device=dev, dtype=torch.bfloat16)
        smq.sparse_mqa_append_kv(self.attn, q, k, v, self.lens, self.cos_sin, slots, workspace=self.ws_attn, q_out=q_rot,
                                 **self.sides())
        smq.sparse_mqa_write_k_cache(self.index, self.randn(rows, DIM), slots, self.k_index, self.ws_index)
        q8 = torch.empty(rows, INDEX_HEADS, DIM, device=dev, dtype=torch.uint8)
        q_scale = torch.empty(rows, device=dev)
        weights = torch.empty(rows, INDEX_HEADS, device=dev, dtype=torch.bfloat16)
        smq.sparse_mqa_quantize_q(self.index, self.randn(rows, INDEX_HEADS, DIM),
                                  torch.randn(rows, INDEX_HEADS, generator=self.generator, device=dev), q8, q_scale, weights)
        self.lens += 1
        ke = self.lens.int()
        candidates = torch.empty(rows, BLOCKS, device=dev, dtype=torch.int32)
        smq.sparse_mqa_candidate_source_decode(self.index, q8, q_scale, weights, self.k_index, self.table, None, ke,
                                               self.longest, candidates, self.ws_source)
        ids = torch.empty(rows, TOPK, device=dev, dtype=torch.int32)
        expansion = torch.empty(rows, self.index.num_sparse_blocks, device=dev, dtype=torch.int32)
        smq.sparse_mqa_logits_topk_decode(self.index, q8, q_scale, weights, self.k_index, self.table, None, ke, candidates,
                                          ids, expansion, torch.empty_like(ke), self.ws_index)
        out, whole = torch.empty_like(q_rot), torch.empty_like(q_rot)
        smq.sparse_mqa_attention_selected(self.attn, q_rot, block_table=self.table, row_indices=None, token_ids=ids, out=out,
                                          workspace=self.ws_attn, **self.sides())
        smq.sparse_mqa_attention_decode(self.attn, q_rot, block_table=self.table, row_indices=None, row_ke=ke, out=whole,
                                        workspace=self.ws_attn, **self.sides())
        for ws in (self.ws_attn, self.ws_index, self.ws_source):
            if smq.smq_get_status(ws):
                raise RuntimeError("a call reported an error")
        return out, whole, ids


def main():
    lens = [300, 1500, 2047, 9000]
    step = Step(lens, longest=9100)
    for n in range(3):
        out, whole, ids = step.run()
        off = (out.float() - whole.float()).norm(dim=(1, 2)) / whole.float().norm(dim=(1, 2))
        print(f"step {n}: selected", (ids >= 0).sum(1).tolist(), "of", step.lens.tolist(),
              "tokens; off the whole context by", [f"{x:.1e}" for x in off.tolist()])


if __name__ == "__main__":
    main()
