"""Plain 64-bit forms of the sequences' attention, what each of its rows sees, and how far a bf16 result of the kernel's
arithmetic can be from them. No code shared with the library."""

import math

import numpy as np
import torch

import attention_ref as ref
import attention_bounds as bounds


def window_sets(n, length, window, sinks):
    """Positions that each of the last n of `length` tokens sees."""
    got = []
    for i in range(n):
        at = length - n + i
        got.append(np.array([t for t in range(max(0, at + 1)) if t < sinks or t > at - window], np.int64))
    return got


def tree_sets(n, length, masks):
    """masks: n sets of node numbers; only nodes below n, at positions that exist, count."""
    base = length - n
    return [np.array(list(range(max(0, base))) + sorted(base + j for j in m if j < n and base + j >= 0), np.int64) for m in masks]


def pack(masks, words):
    bits = np.zeros((len(masks), words * 32), np.uint64)
    for r, m in enumerate(masks):
        for j in m:
            bits[r, j] = 1
    return (bits.reshape(len(masks), words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def random_tree(rng, n):
    """Ancestors of each of n nodes, itself included; every node's parent is an earlier one."""
    got = []
    for j in range(n):
        got.append((set(got[int(rng.integers(max(0, j - 6), j))]) if j else set()) | {j})
    return got


def attend(q, k, v, scale):
    """q [H, D], k and v [tokens, KVH, D] in 64 bits: out, the mean of |v| under the softmax, lse, and the largest sum of
    |q||k| in units of a score of the tokens that have any weight."""
    h, d = q.shape
    if len(k) == 0:
        return np.zeros((h, d)), np.zeros((h, d)), np.full(h, -math.inf), np.zeros(h)
    kvh = k.shape[1]
    qq = q.reshape(kvh, h // kvh, d)
    s = np.einsum("gid,tgd->git", qq, k) * scale
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(-1, keepdims=True)
    lse = (m + np.log(total)).reshape(h)
    w = p / total
    size = np.where(w > 2.0 ** -40, np.einsum("gid,tgd->git", np.abs(qq), np.abs(k)), 0).max(-1).reshape(h) * abs(scale)
    return (np.einsum("git,tgd->gid", w, v).reshape(h, d), np.einsum("git,tgd->gid", w, np.abs(v)).reshape(h, d), lse, size)


def bound(out, mean, size, dim, tokens):
    """The largest error of a bf16 result, and of its lse.

    Scores, sums and joins as in attention_bounds.bound. Weights: one, times its token's value scale, is rounded to bf16, half a
    step: 2^-8 of it. The result is then rounded to the nearest of 8 bits where it is by then: a value below a power of two can
    be above it through what came before, and its half step is twice as long there, so the step is that of |out| plus all
    other errors. Weights below 2^-126 of the largest are zero, and so are results below 2^-126."""
    score = size * (dim / 16 * 17 + 5) * 2.0 ** -24
    moved = (np.expm1(score) + 2.0 ** -21)[:, None]
    off = (np.abs(out) + mean) * moved + mean * (2.0 ** -8 + 8 * math.ceil(tokens / 128) * 17 * 2.0 ** -24 + 2.0 ** -20)
    top = np.maximum(np.abs(out) + off, 2.0 ** -126)
    return off + 2.0 ** (np.floor(np.log2(top)) - 8) + 2.0 ** -100, score + 2.0 ** -20


class Batch:
    """Sequences (rows, length) over one cache, their queries, and the outputs of a call; `pad` rows of no sequence at the end."""

    def __init__(self, rng, heads, kv_heads, dim, page, dtype, seqs, pad=2, scale=None, device="cuda"):
        import sparse_attention_top_expand_gb300 as smq

        self.seqs, self.heads, self.dim, self.device = seqs, heads, dim, device
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        self.cache = ref.Cache(rng, kv_heads, dim, page, dtype, [max(0, length) for _, length in seqs])
        self.order = rng.permutation(len(seqs)).astype(np.int32)  # sequence b reads table row order[b]
        table = np.empty_like(self.cache.table)
        table[self.order] = self.cache.table
        rows = int(self.cu[-1]) + pad
        wide = bounds.bf16(rng.standard_normal((rows, heads * dim + 8)) * 1.5)  # rows a stride apart
        self.q = wide[:, :heads * dim].view(rows, heads, dim).clone()
        self.scale = scale or 1 / math.sqrt(dim)
        self.plan = smq.AttentionPlan(heads, kv_heads, dim, page, max_rows=max(rows, len(seqs), 1), cache_dtype=dtype,
                                      softmax_scale=scale)
        self.table, self.rows = table, rows
        self.workspace = self.plan.sequence_workspace()

    def call(self, sets=None, max_seq_rows=None, **what):
        """Run; `what` is window and sinks, or tree_mask. Tokens that no row of `sets` (per sequence) sees are poisoned."""
        import sparse_attention_top_expand_gb300 as smq

        dev = self.device
        if sets is not None:
            self.poison(sets)
        q = torch.zeros(self.rows, self.heads * self.dim + 8, dtype=torch.bfloat16)
        q[:, :self.heads * self.dim] = self.q.flatten(1)
        self.q_dev = q.to(dev)[:, :self.heads * self.dim].view(self.rows, self.heads, self.dim)
        self.out = torch.full((self.rows, self.heads, self.dim), 9.0, device=dev, dtype=torch.bfloat16)
        self.lse = torch.full((self.rows, self.heads), 9.0, device=dev)
        if "tree_mask" in what:
            what["tree_mask"] = torch.from_numpy(what["tree_mask"]).to(dev)
        longest = max([n for n, _ in self.seqs] + [1])
        self.made = smq.SequenceAttentionCall(
            self.plan, self.q_dev, **self.cache.to(dev), block_table=torch.from_numpy(self.table).to(dev),
            cu_rows=torch.from_numpy(self.cu).to(dev), seq_len=torch.tensor([x for _, x in self.seqs], dtype=torch.int32, device=dev),
            max_seq_rows=max_seq_rows or longest, seq_indices=torch.from_numpy(self.order).to(dev), out=self.out, lse=self.lse,
            workspace=self.workspace, **what)
        self.made()
        return smq.smq_get_status(self.workspace)

    def poison(self, sets):
        """NaN in every token that no row sees, and no page where a whole page is not seen."""
        c = self.cache
        for b, rows in enumerate(sets):
            seen = set(int(t) for s in rows for t in s)
            for col in range(self.table.shape[1]):
                page = int(c.table[b, col])
                unseen = [o for o in range(c.page) if col * c.page + o not in seen]
                if len(unseen) == c.page:
                    self.table[self.order[b], col] = -1
                    continue
                at = torch.tensor(unseen, dtype=torch.long)
                if c.dtype == "bf16":
                    c.data[page, :, :, at] = float("nan")
                else:
                    c.data[page, :, :, at] = 0x7F
                    c.scales[page, :, :, at] = float("nan")

    def check(self, sets, rows=None, skip=()):
        """Compare every row (or `rows` of each sequence) with the plain form over its set."""
        q = self.q.to(torch.float64).numpy()
        out, lse = self.out.to(torch.float64).cpu().numpy(), self.lse.to(torch.float64).cpu().numpy()
        for b, per in enumerate(sets):
            for i, at in enumerate(per):
                r = int(self.cu[b]) + i
                if (rows is not None and i not in rows) or r in skip:
                    continue
                where = f"sequence {b} {self.seqs[b]} row {i}"
                k, v = self.cache.tokens(b, at) if len(at) else (np.zeros((0, 1, self.dim)),) * 2
                want, mean, want_lse, size = attend(q[r], k, v, self.scale)
                off, lse_off = bound(want, mean, size, self.dim, len(at))
                assert np.isfinite(out[r]).all(), f"{where}: not finite"
                if len(at) == 0:
                    assert (out[r] == 0).all() and np.isneginf(lse[r]).all(), f"{where}: a row that sees nothing"
                    continue
                over = np.abs(out[r] - want) - off
                assert (over <= 0).all(), f"{where}: {(over > 0).sum()} of {over.size} over the bound, by {over.max():.3g}"
                over = np.abs(lse[r] - want_lse) - lse_off - 2.0 ** -22 * np.abs(want_lse)
                assert (over <= 0).all(), f"{where}: lse over its bound by {over.max():.3g}"
        assert (out[int(self.cu[-1]):] == 9).all() and (lse[int(self.cu[-1]):] == 9).all(), "rows of no sequence are left alone"

    def window(self, window, sinks=0, poison=True, **kw):
        sets = [window_sets(n, length, window, sinks) for n, length in self.seqs]
        assert self.call(sets if poison else None, window=window, sinks=sinks, **kw) == 0
        self.check(sets)
        return sets

    def tree(self, masks, words=None, **kw):
        """masks: node sets of every row of every sequence, in order."""
        words = words or max(1, -(-max([n for n, _ in self.seqs] + [1]) // 32))
        sets = [tree_sets(n, length, masks[self.cu[b]:self.cu[b] + n]) for b, (n, length) in enumerate(self.seqs)]
        packed = pack(list(masks) + [set(range(words * 32))] * (self.rows - len(masks)), words)
        assert self.call(sets, tree_mask=packed, **kw) == 0
        self.check(sets)
        return sets
