"""Operators around the paged key-value cache, as they are measured: their cases, their inputs, their plain forms.

Two more attentions over the cache, of sequences with one or many query rows each, and the cache's own upkeep:
  window   causal attention with a sliding window and a few first tokens that stay visible
  tree     attention of a tree of drafted tokens over the context and over each token's ancestors
  compact  move a sequence's kept tokens together (the accepted path of a tree, the newer part of a context)
  fork     rows of the block table that share another row's pages, with their own copy of a page begun
  resize   take and release pages, so that rows cover the tokens that they are to hold

`own` chooses what run() does. False: the plain form, in elementary torch operations and 32-bit floats, rounded once
at the end. True: the library's entry points. Both take the same inputs from prepare().

A cache is one allocation, [pages, 2, kv heads, page size, dim] (keys, then values, of a page), of bfloat16, or of E4M3
codes with a float scale for each token, kv head and side. A page is free where its reference count is zero; an entry of
the block table without a page is -1. New pages are the lowest-numbered ones that were free before the call, given out in
the order of rows and columns.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # One new token of one sequence in a sliding layer: the call's latency is what counts.
        dict(name="window_one", op="window", seqs=1, rows_min=1, rows_max=1, heads=64, kv_heads=8, dim=128, page=64, cache="bf16",
             len_min=9000, len_max=9000, window=1024, sinks=4),
        # A decode batch over an 8-bit cache: a token or a few drafted ones for each of 64 sequences, the rows padded.
        dict(name="window_batch_e4m3", op="window", seqs=64, rows_min=1, rows_max=4, heads=64, kv_heads=8, dim=128, page=64,
             cache="e4m3", len_min=4096, len_max=32768, window=4096, sinks=64),
        # A prefill chunk of 4096 tokens of two sequences.
        dict(name="window_chunk", op="window", seqs=2, rows_min=2048, rows_max=2048, heads=64, kv_heads=8, dim=128, page=64,
             cache="bf16", len_min=28672, len_max=36864, window=4096, sinks=4),
        # A tree of eight drafted tokens behind one short context.
        dict(name="tree_one", op="tree", seqs=1, rows_min=8, rows_max=8, heads=64, kv_heads=8, dim=128, page=64, cache="bf16",
             len_min=2047, len_max=2047),
        # Trees of 64 tokens for a batch of 16 sequences: the context has to be read once for many queries.
        dict(name="tree_batch", op="tree", seqs=16, rows_min=64, rows_max=64, heads=64, kv_heads=8, dim=128, page=64, cache="bf16",
             len_min=4096, len_max=32768),
        # Ragged trees, one kv head for all query heads, 64-wide heads, an 8-bit cache.
        dict(name="tree_ragged_e4m3", op="tree", seqs=31, rows_min=5, rows_max=25, heads=32, kv_heads=1, dim=64, page=32,
             cache="e4m3", len_min=100, len_max=16384),
        # After the verification: the accepted path of each of 64 trees moves to the front of its tree.
        dict(name="compact_accepted", op="compact", kind="accepted", rows=64, kv_heads=8, dim=128, page=64, cache="bf16", keep=8,
             nodes=64, len_min=4096, len_max=32768),
        # Contexts that have grown too long: the newer half moves behind the first four tokens, 16 sequences.
        dict(name="compact_newer", op="compact", kind="newer", rows=16, kv_heads=8, dim=128, page=64, cache="bf16", len_min=4096,
             len_max=32768),
        # Eight samples of one prompt.
        dict(name="fork_prompt", op="fork", parents=1, children=8, beams=False, kv_heads=8, dim=128, page=64, cache="bf16",
             len_min=32767, len_max=32767),
        # A beam search's step: 64 groups of 4 beams, each beam's row taken over from one of its group, 8-bit cache.
        dict(name="fork_beams_e4m3", op="fork", parents=64, children=4, beams=True, kv_heads=1, dim=128, page=64, cache="e4m3",
             len_min=100, len_max=32768),
        # A verification step of 64 sequences: room for 64 more tokens, and pages that a window of 4096 has left behind.
        dict(name="resize_step", op="resize", kind="step", rows=64, columns=512, page=64, pages=65536),
        # A batch that turns over: half of 512 sequences end, as many new prompts are admitted.
        dict(name="resize_turnover", op="resize", kind="turnover", rows=512, columns=2048, page=64, pages=524288),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["window", "tree", "window", "tree", "compact", "fork", "resize"])
    page = rng.choice([16, 32, 64, 128, 24])
    if op == "resize":
        kind = rng.choice(["step", "turnover"])
        case = dict(op=op, kind=kind, rows=_log_int(rng, 1, 512), columns=_log_int(rng, 8, 2048), page=page)
        case["pages"] = case["rows"] * case["columns"] // 2 + case["columns"] * 2 + rng.randint(0, 999)
        return case
    kv = rng.choice([1, 1, 2, 4, 8])
    case = dict(op=op, kv_heads=kv, dim=rng.choice([64, 128]), page=page, cache=rng.choice(["bf16", "e4m3"]))
    case["len_max"] = _log_int(rng, 200, 32768)
    case["len_min"] = rng.randint(150, case["len_max"])
    if op == "compact":
        case["kind"] = rng.choice(["accepted", "newer"])
        case["rows"] = _log_int(rng, 1, 64)
        if case["kind"] == "accepted":
            case["keep"] = rng.randint(1, 16)
            case["nodes"] = 2 * case["keep"] + rng.randint(0, 64)
            case["len_min"] = min(case["len_max"], max(case["len_min"], case["nodes"]))
        while case["rows"] * case["len_max"] * kv * case["dim"] > 16 * 18000 * 8 * 128:
            case["rows"] = (case["rows"] + 1) // 2
            case["len_max"] = case["len_max"] // 2 + 150
            case["len_min"] = min(case["len_min"], case["len_max"])
        return case
    if op == "fork":
        case["beams"] = rng.random() < 0.5
        case["children"] = rng.randint(2, 8)
        case["parents"] = _log_int(rng, 1, 64)
        while case["parents"] * case["len_max"] * kv * case["dim"] > 32768 * 8 * 128:
            case["parents"] = (case["parents"] + 1) // 2
            case["len_max"] = case["len_max"] // 2 + 150
            case["len_min"] = min(case["len_min"], case["len_max"])
        return case
    group = min(rng.choice([1, 2, 3, 4, 6, 8, 16, 24, 64, 128]), 128 // kv)
    case["heads"] = kv * group
    case["seqs"] = _log_int(rng, 1, 64)
    case["rows_max"] = _log_int(rng, 1, 1024 if op == "window" else 100)
    case["rows_min"] = rng.randint(1, case["rows_max"])
    if op == "window":
        case["window"] = _log_int(rng, 16, 8192)
        case["sinks"] = rng.choice([0, 0, 1, 4, 64, 130])
    case["len_min"] = max(case["len_min"], case["rows_max"])
    case["len_max"] = max(case["len_max"], case["len_min"])
    while case["seqs"] > 1 and (case["seqs"] * case["len_max"] * kv * case["dim"] > 16 * 18000 * 8 * 128 or work(case)["flops"] > 3e11):
        case["seqs"] = (case["seqs"] + 1) // 2
    while work(case)["flops"] > 3e11:
        case["rows_max"] = (case["rows_max"] + 1) // 2
        case["rows_min"] = min(case["rows_min"], case["rows_max"])
    return case


# ---------------------------------------------------------------- sizes


def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi, so that the work does not depend on the seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _rows(case):
    """The query rows of each sequence: the spread in another order than that of the lengths."""
    r = _spread(case["rows_min"], case["rows_max"], case["seqs"])
    return r[1::2] + r[0::2]


def _first(case, length, rows):
    """The first position that the first of a sequence's rows sees, its sinks apart."""
    return 0 if case["op"] == "tree" else max(0, length - rows + 1 - case["window"])


def _newer(length):
    return max(1, (length - 4) // 2)


def _token(case):
    return case["kv_heads"] * 2 * (2 * case["dim"] if case["cache"] == "bf16" else case["dim"] + 4)


def _fork_columns(case):
    return -(-case["len_max"] // case["page"]) + 1


def _fork_lens(case):
    """The length of every row that a fork makes, and its source row: all beams of all groups, or the children of each parent."""
    lens = _spread(case["len_min"], case["len_max"], case["parents"])
    return [n for n in lens for _ in range(case["children"])]


def _resize_plan(case):
    """Tokens that each row covers now and is to cover: (begin, end) before, (begin, end) after."""
    page, cols = case["page"], case["columns"]
    top = cols * page
    n = case["rows"]
    if case["kind"] == "step":
        lens = _spread(max(1, top // 8), max(1, top - 64), n)
        back = min(4096, top // 2)
        # a window of `back` tokens whose last tidying was three pages ago
        return [(max(0, x - back - 3 * page), x, max(0, x - back), min(top, x + 64)) for x in lens]
    lens = _spread(max(1, top // 64), max(1, top // 2), n)
    return [(0, x, 0, 0) if i % 2 else (0, 0, 0, x) for i, x in enumerate(lens)]


def _pages_of(begin, end, page):
    return max(0, -(-end // page) - begin // page)


def work(case):
    """Bytes and operations of one pass: each input element that is needed read once, each output written once."""
    op = case["op"]
    if op == "resize":
        changed = 0
        for b0, e0, b1, e1 in _resize_plan(case):
            old = set(range(b0 // case["page"], b0 // case["page"] + _pages_of(b0, e0, case["page"])))
            new = set(range(b1 // case["page"], b1 // case["page"] + _pages_of(b1, e1, case["page"])))
            changed += len(old ^ new)
        entries = case["rows"] * case["columns"]
        return {"bytes": 4 * entries + 12 * changed + 8 * case["rows"], "flops": entries}
    if op == "fork":
        entries = len(_fork_lens(case)) * _fork_columns(case)
        copied = sum(n % case["page"] for n in _fork_lens(case))
        shared = sum(n // case["page"] for n in _fork_lens(case))
        return {"bytes": 8 * entries + 8 * shared + 2 * copied * _token(case), "flops": entries}
    if op == "compact":
        if case["kind"] == "accepted":
            kept = sum(_spread(1, case["keep"], case["rows"]))
        else:
            kept = sum(_newer(n) for n in _spread(case["len_min"], case["len_max"], case["rows"]))
        return {"bytes": kept * (2 * _token(case) + 4 + 8), "flops": kept}
    h, d = case["heads"], case["dim"]
    pairs = unique = rows = 0
    for n, r in zip(_spread(case["len_min"], case["len_max"], case["seqs"]), _rows(case)):
        rows += r
        if op == "tree":
            pairs += r * (n - r) + r * 4  # some four ancestors each
            unique += n
        else:
            w, s = case["window"], case["sinks"]
            ends = range(n - r + 1, n + 1)
            pairs += sum(min(e, w) + min(s, max(0, e - w)) for e in ends)
            first = _first(case, n, r)
            unique += n - first + min(s, first)
    return {"bytes": unique * _token(case) + rows * (h * d * 4 + h * 4), "flops": pairs * h * d * 4}


# ---------------------------------------------------------------- inputs


def _quantise(x):
    """x [..., dim] to E4M3 codes (as uint8) and a float scale for each vector: amax / 448, or 1 for zeros."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _cache(s, case, pages, g):
    x = torch.randn(pages, 2, case["kv_heads"], case["page"], case["dim"], generator=g, device=DEVICE, dtype=torch.bfloat16)
    s["cache"], s["scale"] = (x, None) if case["cache"] == "bf16" else _quantise(x)


def _planes(s):
    """What a page holds, as views [pages, heads, page size, ...]."""
    got = [s["cache"][:, 0], s["cache"][:, 1]]
    return got if s["scale"] is None else got + [s["scale"][:, 0], s["scale"][:, 1]]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case=case)
    op, page = case["op"], case["page"]
    if op == "resize":
        return _prepare_resize(s, case, g)
    if op == "fork":
        return _prepare_fork(s, case, g)
    if op == "compact":
        return _prepare_compact(s, case, g)
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    seqs = case["seqs"]
    lens, rows = _spread(case["len_min"], case["len_max"], seqs), _rows(case)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    total = cu[-1] + (3 if seqs > 1 else 0)  # a batch is padded with rows of no sequence
    width = -(-case["len_max"] // page)
    used = torch.zeros(seqs, width, dtype=torch.bool)
    for i, (n, r) in enumerate(zip(lens, rows)):
        used[i, _first(case, n, r) // page : -(-n // page)] = True
        used[i, : -(-min(case.get("sinks", 0), n) // page)] = True  # pages between the sinks and the window are gone
    pages = int(used.sum()) + 1
    order = torch.randperm(pages, generator=g, device=DEVICE).int()
    rank = (torch.cumsum(used.flatten().long(), 0) - 1).view(seqs, width).to(DEVICE)
    s["table"] = torch.where(used.to(DEVICE), order[rank.clamp(min=0)], -1).int().contiguous()
    s["lens"], s["rows"], s["starts"] = lens, rows, cu
    s["cu"] = torch.tensor(cu, device=DEVICE, dtype=torch.int32)
    s["len"] = torch.tensor(lens, device=DEVICE, dtype=torch.int32)
    s["q"] = torch.randn(total, h, d, generator=g, device=DEVICE, dtype=torch.bfloat16) * 1.5
    _cache(s, case, pages, g)
    s["mask"] = None
    if op == "tree":
        most = case["rows_max"]
        words = -(-most // 32)
        seen = torch.zeros(seqs, most, most, dtype=torch.bool)  # node, ancestor or itself
        c = torch.Generator().manual_seed(seed)
        parent = (torch.rand(seqs, most, generator=c) * torch.arange(most)).long()  # an earlier node, the root for node 1
        at = torch.arange(seqs)
        for j in range(most):
            if j:
                seen[:, j] = seen[at, parent[:, j]]
            seen[:, j, j] = True
        bits = torch.zeros(seqs, most, words * 32, dtype=torch.int64)
        bits[:, :, :most] = seen.long()
        packed = (bits.view(seqs, most, words, 32) << torch.arange(32)).sum(-1)
        packed = torch.where(packed >= 2**31, packed - 2**32, packed).int()
        mask = torch.zeros(total, words, dtype=torch.int32)
        for i, r in enumerate(rows):
            mask[cu[i] : cu[i] + r] = packed[i, :r]
        s["mask"] = mask.to(DEVICE)
    # one row more than the call has takes what the plain form computes for rows that are not there
    s["room"] = torch.zeros(total + 1, h, d, device=DEVICE, dtype=torch.bfloat16), torch.zeros(total + 1, h, device=DEVICE)
    s["out"], s["lse"] = (x[:total] for x in s["room"])
    if own:  # the handle that a program keeps: the plan, its workspace and the call with its arguments marshalled
        import sparse_attention_top_expand_gb300 as smq

        plan = smq.AttentionPlan(num_heads=h, num_kv_heads=kv, head_dim=d, page_size=page, max_rows=total, cache_dtype=case["cache"])
        cache, scale = s["cache"], s["scale"]
        what = dict(window=case["window"], sinks=case["sinks"]) if op == "window" else dict(tree_mask=s["mask"])
        s["call"] = smq.SequenceAttentionCall(
            plan, s["q"], cache[:, 0], cache[:, 1], s["table"], s["cu"], s["len"], case["rows_max"], s["out"],
            plan.sequence_workspace(), lse=s["lse"], k_scales=None if scale is None else scale[:, 0],
            v_scales=None if scale is None else scale[:, 1], **what)
    return s


def _flat(s, refs, table):
    """Reference counts and block table in one buffer, and a copy of what they were before a pass."""
    s["flat"] = torch.cat([refs.flatten(), table.flatten()]).int().to(DEVICE)
    s["before"] = s["flat"].clone()
    s["refs"] = s["flat"][: refs.numel()]
    s["table"] = s["flat"][refs.numel() :].view(table.shape)


def _prepare_resize(s, case, g):
    rows, cols, page, pages = case["rows"], case["columns"], case["page"], case["pages"]
    plan = torch.tensor(_resize_plan(case))
    plan = plan[torch.randperm(rows, generator=g, device=DEVICE).cpu()]
    col = torch.arange(cols)
    held = (col >= plan[:, :1] // page) & (col < (plan[:, 1:2] + page - 1) // page)
    order = torch.randperm(pages, generator=g, device=DEVICE).cpu()
    rank = torch.cumsum(held.flatten().long(), 0).view(rows, cols) - 1
    table = torch.where(held, order[rank.clamp(min=0)], -1)
    refs = torch.zeros(pages, dtype=torch.int64)
    refs[table[held]] = 1
    if case["kind"] == "turnover":  # prompts that other rows still hold keep their pages
        lucky = order[: int(held.sum())][::7]
        refs[lucky] += 1
    _flat(s, refs, table)
    s["begin"], s["end"] = (plan[:, i].int().to(DEVICE).contiguous() for i in (2, 3))
    if own:
        import sparse_attention_top_expand_gb300 as smq

        plan = smq.PagePlan(page_size=page, num_pages=pages, table_rows=rows, table_columns=cols)
        s["call"] = smq.ResizeCall(plan, s["refs"], s["table"], s["end"], plan.workspace(), row_begin=s["begin"])
    return s


def _prepare_fork(s, case, g):
    page, cols = case["page"], _fork_columns(case)
    per, groups = case["children"], case["parents"]
    lens = _spread(case["len_min"], case["len_max"], groups)
    holders = per if case["beams"] else 1  # rows that hold a group's pages before the call
    rows = groups * per if case["beams"] else groups * (1 + per)
    need = sum(n // page + holders * (n % page > 0) for n in lens)
    pages = need + groups * per + 64
    order = torch.randperm(pages, generator=g, device=DEVICE).cpu()
    table = torch.full((rows, cols), -1, dtype=torch.int64)
    refs = torch.zeros(pages, dtype=torch.int64)
    src, dst, at = [], [], 0
    pick = torch.randint(0, per, (groups, per), generator=g, device=DEVICE).cpu().tolist()
    for i, n in enumerate(lens):
        full, first = n // page, i * per if case["beams"] else i * (1 + per)
        for b in range(holders):  # a prompt's whole pages are shared, the page begun is each beam's own
            table[first + b, :full] = order[at : at + full]
            if n % page:
                table[first + b, full] = order[at + full + b]
                refs[order[at + full + b]] = 1
        refs[order[at : at + full]] = holders
        at += full + holders * (n % page > 0)
        for b in range(per):
            src.append(first + pick[i][b] if case["beams"] else first)
            dst.append(first + b if case["beams"] else first + 1 + b)
    _flat(s, refs, table)
    s["src"], s["dst"], s["len"] = (torch.tensor(x, device=DEVICE, dtype=torch.int32) for x in (src, dst, _fork_lens(case)))
    _cache(s, case, pages, g)
    if own:
        import sparse_attention_top_expand_gb300 as smq

        plan = smq.PagePlan(page_size=page, num_pages=pages, table_rows=rows, table_columns=cols)
        s["call"] = smq.ForkCall(plan, s["refs"], s["table"], s["src"], s["dst"], s["len"], _planes(s), plan.workspace())
    return s


def _prepare_compact(s, case, g):
    page, rows = case["page"], case["rows"]
    lens = _spread(case["len_min"], case["len_max"], rows)
    width = -(-case["len_max"] // page)
    need = torch.tensor([-(-n // page) for n in lens])
    pages = int(need.sum()) + 1
    order = torch.randperm(pages, generator=g, device=DEVICE).cpu()
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width)
    used = col < need.unsqueeze(1)
    table = torch.where(used, order[(first.unsqueeze(1) + col).clamp(max=pages - 1)], -1)
    refs = torch.zeros(pages, dtype=torch.int64)
    refs[table[used]] = 1
    s["refs"], s["table"] = refs.int().to(DEVICE), table.int().to(DEVICE).contiguous()
    # Kept tokens that move come from behind the places that they move to, so that a pass can be repeated.
    start, ids = [], []
    if case["kind"] == "accepted":
        for n, k in zip(lens, _spread(1, case["keep"], rows)):
            path = torch.randperm(case["nodes"] - case["keep"], generator=g, device=DEVICE)[: k - 1].sort().values.cpu() + case["keep"]
            start.append(n - case["nodes"])
            ids.append([n - case["nodes"]] + (n - case["nodes"] + path).tolist())  # the root stays where it is
    else:
        for n in lens:
            k = _newer(n)
            start.append(4)
            ids.append(range(n - k, n))
    most = max(len(x) for x in ids)
    keep = torch.full((rows, most), -1, dtype=torch.int32)
    for i, x in enumerate(ids):
        keep[i, : len(x)] = torch.tensor(list(x), dtype=torch.int32)
    s["start"], s["keep"] = torch.tensor(start, device=DEVICE, dtype=torch.int32), keep.to(DEVICE)
    _cache(s, case, pages, g)
    if own:
        import sparse_attention_top_expand_gb300 as smq

        plan = smq.PagePlan(page_size=page, num_pages=pages, table_rows=rows, table_columns=width)
        s["call"] = smq.CompactCall(plan, s["refs"], s["table"], s["start"], s["keep"], _planes(s), plan.workspace())
    return s


# ---------------------------------------------------------------- plain forms


def _values(s, page, off):
    """Keys and values of tokens at (page, off) [sequences, tokens] as floats [sequences, kv heads, tokens, dim]."""
    got = []
    for side in (0, 1):
        x = s["cache"][:, side][page, :, off]
        if s["scale"] is None:
            x = x.float()
        else:
            x = x.view(torch.float8_e4m3fn).float() * s["scale"][:, side][page, :, off].unsqueeze(-1)
        got.append(x.transpose(1, 2))
    return got


def _attention_block(s, seqs, i0, i1):
    """Rows i0 .. i1 of the given sequences, together: gather what any of them sees, and mask the scores."""
    case = s["case"]
    page, h, kv, d = case["page"], case["heads"], case["kv_heads"], case["dim"]
    pick = torch.tensor(seqs, device=DEVICE)
    length, first_row = s["len"][pick].long(), s["cu"][pick].long()
    rows = s["cu"][pick + 1].long() - first_row
    i = torch.arange(i0, i1, device=DEVICE)
    there = i < rows.unsqueeze(1)
    index = torch.where(there, first_row.unsqueeze(1) + i, s["room"][0].shape[0] - 1)
    longest = max(s["lens"][x] for x in seqs)
    if case["op"] == "tree":
        at = torch.arange(longest, device=DEVICE).expand(len(seqs), -1)
        node = at - (length - rows).unsqueeze(1)
        mask = s["mask"][torch.where(there, index, 0)].long()
        word = (node // 32).clamp(0, mask.shape[-1] - 1)
        bit = (mask.gather(2, word.unsqueeze(1).expand(-1, len(i), -1)) >> (node % 32).unsqueeze(1)) & 1
        valid = (at < length.unsqueeze(1)).unsqueeze(1) & ((node < 0).unsqueeze(1) | (bit == 1))
    else:
        end = (length - rows).unsqueeze(1) + i + 1
        low = min(max(0, s["lens"][x] - s["rows"][x] + i0 + 1 - case["window"]) for x in seqs)
        start = (end[:, :1] - case["window"]).clamp(min=0)
        span = min(longest - low, case["window"] + i1 - i0)
        sinks = torch.arange(case["sinks"], device=DEVICE).expand(len(seqs), -1)
        band = start + torch.arange(span, device=DEVICE)
        at = torch.cat([sinks, band], 1)
        new = torch.cat([sinks < start, torch.ones_like(band, dtype=torch.bool)], 1)  # sinks that the band has not
        seen = (at.unsqueeze(1) >= (end - case["window"]).unsqueeze(2)) | (at < case["sinks"]).unsqueeze(1)
        valid = new.unsqueeze(1) & (at.unsqueeze(1) < end.unsqueeze(2)) & seen
    valid = valid & there.unsqueeze(2)
    col = (at // page).clamp(max=s["table"].shape[1] - 1)
    k, v = _values(s, s["table"][pick].long().gather(1, col).clamp(min=0), at % page)
    q = s["q"][torch.where(there, index, 0)].float().view(len(seqs), len(i), kv, h // kv, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(len(seqs), kv, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)).view(len(seqs), kv, len(i), h // kv, -1) * (1.0 / math.sqrt(d))
    score = score.masked_fill(~valid[:, None, :, None, :], -math.inf)
    most = score.amax(-1, keepdim=True)
    most = torch.where(most > -math.inf, most, torch.zeros_like(most))
    p = torch.exp(score - most)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(len(seqs), kv, -1, p.shape[-1]), v).view(len(seqs), kv, len(i), h // kv, d)
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    s["room"][0][index] = out.permute(0, 2, 1, 3, 4).reshape(len(seqs), len(i), h, d).bfloat16()
    s["room"][1][index] = (most + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(len(seqs), len(i), h)


def _attention_plain(s):
    case = s["case"]
    step = min(case["rows_max"], 256)
    seen = case["len_max"] if case["op"] == "tree" else min(case["len_max"], case["window"] + step) + case["sinks"]
    each = seen * (case["heads"] * step * 4 * 4 + case["kv_heads"] * case["dim"] * 16)  # bytes of a sequence's block
    batch = max(1, int(24e9 // each))
    for a in range(0, case["seqs"], batch):
        seqs = list(range(a, min(case["seqs"], a + batch)))
        for i0 in range(0, max(s["rows"][x] for x in seqs), step):
            _attention_block(s, seqs, i0, i0 + step)


def _resize_plain(s):
    case, table, refs = s["case"], s["table"], s["refs"]
    col = torch.arange(case["columns"], device=DEVICE)
    page = case["page"]
    wanted = (col >= (s["begin"] // page).unsqueeze(1)) & (col < ((s["end"] + page - 1) // page).unsqueeze(1))
    has = table >= 0
    take, drop = wanted & ~has, has & ~wanted
    free = torch.nonzero(refs == 0).squeeze(1)
    refs.index_add_(0, table[drop].long(), torch.full((1,), -1, device=DEVICE, dtype=torch.int32).expand(int(drop.sum())))
    table[drop] = -1
    got = free[: int(take.sum())]
    table[take] = got.int()
    refs[got] = 1


def _fork_plain(s):
    case, table, refs, page = s["case"], s["table"], s["refs"], s["case"]["page"]
    src, dst, length = s["src"].long(), s["dst"].long(), s["len"].long()
    moves = src != dst  # a row forked onto itself stays as it is
    src, dst, length = src[moves], dst[moves], length[moves]
    old, row = table[dst], table[src]
    col = torch.arange(table.shape[1], device=DEVICE)
    full = (length // page).unsqueeze(1)
    share = (col < full) & (row >= 0)
    begun = row.gather(1, full).squeeze(1).long()
    take = (length % page > 0) & (begun >= 0)
    free = torch.nonzero(refs == 0).squeeze(1)[: int(take.sum())]
    one = torch.ones(1, device=DEVICE, dtype=torch.int32)
    refs.index_add_(0, row[share].long(), one.expand(int(share.sum())))
    refs[free] = 1
    drop = old >= 0
    refs.index_add_(0, old[drop].long(), (-one).expand(int(drop.sum())))
    new = torch.where(share, row, -1)
    fresh = torch.full_like(length, -1)
    fresh[take] = free
    new.scatter_(1, full, torch.where(take, fresh, -1).int().unsqueeze(1))
    table[dst] = new
    keep = torch.arange(page, device=DEVICE) < (length[take] % page).unsqueeze(1)
    for plane in _planes(s):
        a, b = plane[begun[take]], plane[free]
        plane[free] = torch.where(keep.view(len(keep), 1, page, *[1] * (plane.dim() - 3)), a, b)


def _compact_plain(s):
    page, table, keep = s["case"]["page"], s["table"], s["keep"].long()
    row, j = torch.nonzero(keep >= 0, as_tuple=True)
    src, dst = keep[row, j], s["start"].long()[row] + j
    a, b = table[row, src // page].long(), table[row, dst // page].long()
    for plane in _planes(s):
        plane[b, :, dst % page] = plane[a, :, src % page]


def run(s):
    op = s["case"]["op"]
    if op in ("resize", "fork"):
        s["flat"].copy_(s["before"])  # what a program has before the call
    if own:
        s["call"]()
    else:
        {"window": _attention_plain, "tree": _attention_plain, "compact": _compact_plain, "fork": _fork_plain,
         "resize": _resize_plain}[op](s)
    return _outputs(s)


def _outputs(s):
    op = s["case"]["op"]
    if op in ("window", "tree"):
        return {"out": s["out"], "lse": s["lse"]}
    got = {} if op == "compact" else {"table": s["table"], "refs": s["refs"]}
    if op != "resize":
        got["cache"] = s["cache"] if s["scale"] is None else s["cache"].view(torch.float8_e4m3fn)
        if s["scale"] is not None:
            got["scale"] = s["scale"]
    return got


# ---------------------------------------------------------------- exact results


def _exact_attention(s, case):
    h, kv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    total = s["out"].shape[0]
    out = torch.zeros(total, h, d, device=DEVICE, dtype=torch.float64)
    lse = torch.zeros(total, h, device=DEVICE, dtype=torch.float64)
    cu, lens, table = s["cu"].tolist(), s["len"].tolist(), s["table"].cpu()
    bits = None if s["mask"] is None else (s["mask"].cpu().numpy().view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32) & 1)
    for b, n in enumerate(lens):
        for r0 in range(cu[b], cu[b + 1], 128):
            r1 = min(cu[b + 1], r0 + 128)
            see = torch.zeros(r1 - r0, n, dtype=torch.bool)
            for r in range(r0, r1):
                behind = cu[b + 1] - r  # rows from this one to the last
                if case["op"] == "tree":
                    base = n - (cu[b + 1] - cu[b])
                    see[r - r0, :base] = True
                    see[r - r0, base:] = torch.from_numpy(bits[r].reshape(-1)[: n - base].astype(bool))
                else:
                    end = n - behind + 1
                    see[r - r0, max(0, end - case["window"]) : end] = True
                    see[r - r0, : min(case["sinks"], end)] = True
            at = torch.nonzero(see.any(0)).squeeze(1)
            see = see[:, at].to(DEVICE)
            where, off = table[b].long()[at // page].to(DEVICE), (at % page).to(DEVICE)
            x = s["cache"][where, :, :, off]  # [tokens, 2, kv heads, dim]
            if s["scale"] is None:
                x = x.double()
            else:
                x = x.view(torch.float8_e4m3fn).double() * s["scale"][where, :, :, off].double().unsqueeze(-1)
            for e in range(kv):
                heads = slice(e * (h // kv), (e + 1) * (h // kv))
                y = torch.einsum("rgd,td->rgt", s["q"][r0:r1, heads].double(), x[:, 0, e]) / math.sqrt(d)
                y.masked_fill_(~see.unsqueeze(1), -math.inf)
                lse[r0:r1, heads] = torch.logsumexp(y, -1)
                out[r0:r1, heads] = torch.einsum("rgt,td->rgd", torch.softmax(y, -1), x[:, 1, e])
    return {"out": out, "lse": lse}


def exact(case, seed):
    """The outputs in 64 bits, row by row; tables, counts and moved tokens entry by entry on the host."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("window", "tree"):
        return _exact_attention(s, case)
    page = case["page"]
    table, refs = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    moves = []  # (from page, its tokens, to page, its tokens)
    if op == "resize":
        free = iter(np.flatnonzero(refs == 0).tolist())
        for r, (b, e) in enumerate(zip(s["begin"].tolist(), s["end"].tolist())):
            lo, hi = b // page, -(-e // page)
            row = table[r]
            for c in np.flatnonzero(row >= 0):
                if not lo <= c < hi:
                    refs[row[c]] -= 1
                    row[c] = -1
            for c in range(lo, hi):
                if row[c] < 0:
                    row[c] = next(free)
                    refs[row[c]] += 1
    elif op == "fork":
        was, free = table.copy(), iter(np.flatnonzero(refs == 0).tolist())
        for a, b, n in zip(s["src"].tolist(), s["dst"].tolist(), s["len"].tolist()):
            if a == b:
                continue
            table[b] = -1
            for c in range(-(-n // page)):
                if was[a, c] >= 0 and (c + 1) * page <= n:
                    table[b, c] = was[a, c]
                elif was[a, c] >= 0:
                    table[b, c] = next(free)
                    moves.append((was[a, c], np.arange(n - c * page), table[b, c], np.arange(n - c * page)))
                if table[b, c] >= 0:
                    refs[table[b, c]] += 1
            for x in was[b][was[b] >= 0]:
                refs[x] -= 1
    else:
        for r, (first, ids) in enumerate(zip(s["start"].tolist(), s["keep"].tolist())):
            a = np.array([i for i in ids if i >= 0])
            b = first + np.arange(len(a))
            moves.append((table[r][a // page], a % page, table[r][b // page], b % page))
    got = dict(_outputs(s))
    if op != "compact":
        got["table"], got["refs"] = torch.from_numpy(table).to(DEVICE), torch.from_numpy(refs).to(DEVICE)
    if op != "resize":
        for name in [x for x in ("cache", "scale") if x in got]:
            new = got[name].clone()
            for a, ta, b, tb in moves:
                a, ta, b, tb = (torch.as_tensor(np.asarray(x, np.int64)).to(DEVICE) for x in (a, ta, b, tb))
                new[b, :, :, tb] = got[name][a, :, :, ta]
            got[name] = new.double() if name == "cache" else new
    return got
