"""The attention operators that follow the indexer, as they are measured: their cases, their inputs, their plain forms.

Three operators share one paged key-value cache:
  append    rotate a step's queries and keys by their positions and write keys and values into the cache
  decode    attention of one query row over its whole cached context
  selected  attention of one query row over the token ids that the indexer selected

`own` chooses what run() does. False: the plain form, in elementary torch operations and 32-bit floats, rounded once
at the end. True: the library's entry points. Both take the same inputs from prepare().

The cache is one allocation, [pages, 2, kv heads, page size, dim] (keys, then values, of a page), so a page of keys and a
page of values are strided views. It holds bfloat16, or E4M3 codes with a float scale for each token, kv head and side.
"""

import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 128  # candidate block size of the indexer, in tokens


def listed():
    return [
        # One new token of one sequence joins the cache: the call's latency is what counts.
        dict(name="append_one", op="append", rows=1, heads=64, kv_heads=1, dim=128, rot=64, pairs="half", page=64, cache="bf16"),
        # The new tokens of a decode batch, 64 sequences, eight kv heads, into an 8-bit cache.
        dict(name="append_step_e4m3", op="append", rows=64, heads=64, kv_heads=8, dim=128, rot=128, pairs="half", page=64, cache="e4m3"),
        # A prefill chunk of 4096 tokens: its queries are rotated and its keys and values appended.
        dict(name="append_chunk", op="append", rows=4096, heads=64, kv_heads=8, dim=128, rot=128, pairs="half", page=64, cache="bf16"),
        # A ragged chunk with interleaved rotation pairs and 64-wide heads into an 8-bit cache.
        dict(name="append_chunk_e4m3", op="append", rows=4093, heads=32, kv_heads=4, dim=64, rot=64, pairs="interleaved", page=32,
             cache="e4m3"),
        # A few short contexts, one of them empty: latency.
        dict(name="decode_short", op="decode", rows=8, heads=64, kv_heads=8, dim=64, page=64, cache="bf16", len_min=0, len_max=2047),
        # One sequence with a long context: the work has to be split over its length.
        dict(name="decode_one_long", op="decode", rows=1, heads=64, kv_heads=1, dim=128, page=64, cache="bf16", len_min=131071,
             len_max=131071),
        # The decode batch, contexts of 4096 to 32768 tokens, eight query heads on each of eight kv heads.
        dict(name="decode_batch", op="decode", rows=64, heads=64, kv_heads=8, dim=128, page=64, cache="bf16", len_min=4096, len_max=32768),
        # The same batch with one kv head for all 64 query heads and an 8-bit cache.
        dict(name="decode_batch_e4m3", op="decode", rows=64, heads=64, kv_heads=1, dim=128, page=64, cache="e4m3", len_min=4096,
             len_max=32768),
        # A row of the tiny configuration's kind: 64 selected tokens out of contexts of up to 1024.
        dict(name="selected_tiny", op="selected", rows=4, heads=8, kv_heads=1, dim=128, page=64, cache="bf16", len_min=40, len_max=1024,
             topk=64, seqs=4),
        # The decode batch behind the indexer: 2048 selected tokens for each of 64 rows.
        dict(name="selected_batch", op="selected", rows=64, heads=64, kv_heads=1, dim=128, page=64, cache="bf16", len_min=4096,
             len_max=32768, topk=2048, seqs=64),
        # The long-context batch: 256 rows, short ones among them (their ids are padded with -1), 8-bit cache.
        dict(name="selected_long_e4m3", op="selected", rows=256, heads=64, kv_heads=1, dim=128, page=64, cache="e4m3", len_min=1,
             len_max=65535, topk=2048, seqs=256),
        # A prefill chunk: 4096 rows of two sequences, 2048 selected tokens each.
        dict(name="selected_chunk", op="selected", rows=4096, heads=64, kv_heads=1, dim=128, page=64, cache="bf16", len_min=28672,
             len_max=36864, topk=2048, seqs=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "decode", "selected"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16, 24, 64, 128])
    group = min(group, 128 // kv)
    case = dict(op=op, rows=0, heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]))
    if op == "append":
        case["rows"] = _log_int(rng, 1, 4096)
        case["rot"] = rng.choice([dim, dim // 2])
        case["pairs"] = rng.choice(["half", "interleaved"])
        return case
    case["len_max"] = _log_int(rng, 16, 131072)
    if op == "decode":
        case["rows"] = _log_int(rng, 1, 256)
        case["len_min"] = rng.randint(0, case["len_max"])
        while case["rows"] * case["len_max"] * kv * dim > 64 * 32768 * 8 * 128 // 2 or work(case)["flops"] > 2.5e11:
            case["rows"] = (case["rows"] + 1) // 2
            case["len_max"] = case["len_max"] // 2 + 1
            case["len_min"] = min(case["len_min"], case["len_max"])
        return case
    case["topk"] = _log_int(rng, 16, 2048)
    case["rows"] = _log_int(rng, 1, 2048)
    case["seqs"] = rng.choice([case["rows"], max(1, case["rows"] // 16)])
    case["len_min"] = rng.randint(1, case["len_max"])
    while case["rows"] * case["topk"] * kv * dim > 4096 * 2048 * 128 or work(case)["flops"] > 2.5e11:
        case["rows"] = (case["rows"] + 1) // 2
    case["seqs"] = min(case["seqs"], case["rows"])
    while case["seqs"] * case["len_max"] * kv * dim > 64 * 32768 * 8 * 128 // 2:
        case["len_max"] = case["len_max"] // 2 + 1
        case["len_min"] = min(case["len_min"], case["len_max"])
    return case


def _lengths(case):
    """The context lengths of a case, evenly spread, so that the work does not depend on the seed."""
    n = case.get("seqs", case["rows"])
    lo, hi = case["len_min"], case["len_max"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def work(case):
    """Bytes and operations of one pass: each input element that is needed read once, each output written once."""
    h, kv, d, rows = case["heads"], case["kv_heads"], case["dim"], case["rows"]
    token = kv * 2 * (2 * d if case["cache"] == "bf16" else d + 4)  # bytes of one token's keys and values
    if case["op"] == "append":
        read = rows * ((h + 2 * kv) * d * 2 + 8 + 8 + case["rot"] * 4)
        return {"bytes": read + rows * (h * d * 2 + token), "flops": rows * (h + kv) * case["rot"] * 3}
    lens = _lengths(case)
    if case["op"] == "decode":
        pairs, unique = sum(lens), sum(lens)
    else:
        per = rows // len(lens)
        valid = [min(case["topk"], n) for n in lens]
        count = [per + (1 if i < rows % len(lens) else 0) for i in range(len(lens))]
        pairs = sum(c * v for c, v in zip(count, valid))
        unique = sum(min(n, c * v) for c, v, n in zip(count, valid, lens))
    other = rows * (h * d * 4 + h * 4) + (pairs * 4 if case["op"] == "selected" else 4 * rows)
    return {"bytes": unique * token + other, "flops": pairs * h * d * 4}


def _quantise(x):
    """x [..., dim] to E4M3 codes (as uint8) and a float scale for each vector: amax / 448, or 1 for zeros."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    h, kv, d, page, rows = case["heads"], case["kv_heads"], case["dim"], case["page"], case["rows"]
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.bfloat16)

    if case["op"] == "append":
        pages = -(-rows // page) + 3
        slots = torch.randperm(pages * page, generator=g, device=DEVICE)[:rows]
        if rows > 1:
            slots[rows // 2] = -1  # a padding token
        s["slots"] = slots
        positions = 32768
        s["positions"] = torch.randint(0, positions, (rows,), generator=g, device=DEVICE)
        half = case["rot"] // 2
        angle = torch.arange(positions, device=DEVICE).float().unsqueeze(1) * torch.exp(
            torch.arange(half, device=DEVICE).float() * (-math.log(10000.0) / half))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        qkv = randn(rows, (h + 2 * kv) * d)  # a fused projection: queries, keys and values are views of its rows
        s["q"] = qkv[:, : h * d].view(rows, h, d)
        s["k"] = qkv[:, h * d : (h + kv) * d].view(rows, kv, d)
        s["v"] = qkv[:, (h + kv) * d :].view(rows, kv, d)
        s["q_out"] = torch.empty(rows, h, d, device=DEVICE, dtype=torch.bfloat16)
        if case["cache"] == "bf16":
            s["cache"] = torch.zeros(pages, 2, kv, page, d, device=DEVICE, dtype=torch.bfloat16)
            s["scale"] = None
        else:
            s["cache"] = torch.zeros(pages, 2, kv, page, d, device=DEVICE, dtype=torch.uint8)
            s["scale"] = torch.ones(pages, 2, kv, page, device=DEVICE)
    else:
        lens = _lengths(case)
        seqs = len(lens)
        lens = torch.tensor(lens, device=DEVICE)[torch.randperm(seqs, generator=g, device=DEVICE)] if case["op"] == "decode" else \
            torch.tensor(lens, device=DEVICE)
        width = max(1, -(-case["len_max"] // page))
        need = (lens + page - 1) // page
        pages = int(need.sum()) + 1
        order = torch.randperm(pages, generator=g, device=DEVICE).int()
        first = torch.cumsum(need, 0) - need
        col = torch.arange(width, device=DEVICE)
        used = col < need.unsqueeze(1)
        # entries past a sequence's last page are left over from other sequences: valid pages, not read
        s["table"] = order[torch.where(used, first.unsqueeze(1) + col, col % pages)].contiguous()
        s["index"] = (torch.arange(rows, device=DEVICE) % seqs).int()
        s["q"] = randn(rows, h, d) * 1.5
        cache = randn(pages, 2, kv, page, d)
        s["scale"] = None
        if case["cache"] == "e4m3":
            cache, s["scale"] = _quantise(cache)
        s["cache"] = cache
        if case["op"] == "decode":
            s["len"] = lens.int()
        else:
            # what the indexer publishes: the better half of the positions in a row's candidate blocks, best first
            topk, blocks = case["topk"], -(-case["len_max"] // BLOCK)
            context = lens[s["index"].long()].unsqueeze(1)
            score = torch.rand(rows, blocks, generator=g, device=DEVICE)
            score = torch.where(torch.arange(blocks, device=DEVICE) * BLOCK < context, score, -1.0)
            chosen = score.topk(min(blocks, -(-2 * topk // BLOCK) + 1), 1).indices
            at = (chosen.unsqueeze(2) * BLOCK + torch.arange(BLOCK, device=DEVICE)).flatten(1)
            score = torch.where(at < context, torch.rand(at.shape, generator=g, device=DEVICE), -1.0)
            best = score.topk(min(topk, at.shape[1]), 1)
            ids = torch.full((rows, topk), -1, device=DEVICE, dtype=torch.int32)
            ids[:, : best.indices.shape[1]] = torch.where(best.values >= 0, at.gather(1, best.indices), -1).int()
            s["ids"] = ids
        s["out"] = torch.empty(rows, h, d, device=DEVICE, dtype=torch.bfloat16)
        s["lse"] = torch.empty(rows, h, device=DEVICE)
    if own:  # the handle that a program keeps: the plan, its workspace and the call with its arguments marshalled
        import sparse_attention_top_expand_gb300 as smq

        plan = smq.AttentionPlan(num_heads=h, num_kv_heads=kv, head_dim=d, page_size=page, max_rows=rows, cache_dtype=case["cache"])
        cache, scale = s["cache"], s["scale"]
        sides = dict(k_cache=cache[:, 0], v_cache=cache[:, 1], k_scales=None if scale is None else scale[:, 0],
                     v_scales=None if scale is None else scale[:, 1], workspace=plan.workspace())
        if case["op"] == "append":
            s["call"] = smq.AppendCall(plan, s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], q_out=s["q_out"],
                                       interleaved=case["pairs"] == "interleaved", **sides)
        elif case["op"] == "decode":
            s["call"] = smq.AttentionCall(plan, s["q"], block_table=s["table"], row_indices=s["index"], row_ke=s["len"], out=s["out"],
                                          lse=s["lse"], **sides)
        else:
            s["call"] = smq.AttentionCall(plan, s["q"], block_table=s["table"], row_indices=s["index"], token_ids=s["ids"],
                                          out=s["out"], lse=s["lse"], **sides)
    return s


def _rotate(x, table, pairs):
    """x [rows, heads, dim] rotated in 32 bits by table [rows, rot] (cosines, then sines)."""
    half = table.shape[1] // 2
    c, n = table[:, None, :half], table[:, None, half:]
    x = x.float()
    if pairs == "half":
        a, b = x[..., :half], x[..., half : 2 * half]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = x[..., : 2 * half : 2], x[..., 1 : 2 * half : 2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half :]], -1)


def _append_plain(s):
    case, page = s["case"], s["case"]["page"]
    table = s["cos_sin"][s["positions"]]
    s["q_out"].copy_(_rotate(s["q"], table, case["pairs"]).bfloat16())
    k, v = _rotate(s["k"], table, case["pairs"]), s["v"].float()
    keep = torch.nonzero(s["slots"] >= 0).squeeze(1)
    slot = s["slots"][keep]
    at = (slot // page, slice(None), slot % page)
    for side, x in enumerate((k[keep], v[keep])):
        if s["scale"] is None:
            s["cache"][:, side][at] = x.bfloat16()
        else:
            code, scale = _quantise(x)
            s["cache"][:, side][at] = code
            s["scale"][:, side][at] = scale


def _softmax_plain(s, k, v, valid):
    """Attention of q [rows, heads, dim] over k, v [rows, kv heads, tokens, dim] in 32 bits where valid [rows, tokens]."""
    rows, h, d = s["q"].shape
    kv = k.shape[1]
    q = s["q"].float().view(rows, kv, h // kv, d)
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    score = score.masked_fill(~valid[:, None, None, :], -math.inf)
    most = score.amax(-1, keepdim=True)
    most = torch.where(most > -math.inf, most, torch.zeros_like(most))
    p = torch.exp(score - most)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(out.view(rows, h, d).bfloat16())
    s["lse"].copy_((most + torch.log(total)).view(rows, h))


def _sides_plain(s, page, off):
    """Keys and values of tokens at (page, off) [rows, tokens] as floats [rows, kv heads, tokens, dim]."""
    got = []
    for side in (0, 1):
        x = s["cache"][:, side][page, :, off]
        if s["scale"] is None:
            x = x.float()
        else:
            x = x.view(torch.float8_e4m3fn).float() * s["scale"][:, side][page, :, off].unsqueeze(-1)
        got.append(x.transpose(1, 2))
    return got


def _decode_plain(s):
    page = s["case"]["page"]
    table = s["table"][s["index"].long()].long()
    at = torch.arange(table.shape[1] * page, device=DEVICE)
    valid = at < s["len"][s["index"].long()].unsqueeze(1)
    k, v = _sides_plain(s, table[:, at // page], (at % page).expand(table.shape[0], -1))
    _softmax_plain(s, k, v, valid)


def _selected_plain(s):
    page = s["case"]["page"]
    valid = s["ids"] >= 0
    at = torch.where(valid, s["ids"], 0).long()
    table = s["table"][s["index"].long()].long()
    k, v = _sides_plain(s, table.gather(1, at // page), at % page)
    _softmax_plain(s, k, v, valid)


def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    else:
        {"append": _append_plain, "decode": _decode_plain, "selected": _selected_plain}[op](s)
    if op == "append":
        if s["scale"] is None:
            return {"q": s["q_out"], "cache": s["cache"]}
        return {"q": s["q_out"], "cache": s["cache"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    return {"out": s["out"], "lse": s["lse"]}


def exact(case, seed):
    """The outputs in 64 bits, row by row. An 8-bit cache has no exact value of its own after a rounding: None there."""
    s = prepare(case, seed)
    rows, h, kv, d, page = case["rows"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        half = case["rot"] // 2
        first = torch.arange(half, device=DEVICE)
        first, second = (first, first + half) if case["pairs"] == "half" else (2 * first, 2 * first + 1)
        turn = s["cos_sin"].double()[s["positions"]]
        phase = torch.complex(turn[:, :half], turn[:, half:]).unsqueeze(1)

        def rotated(x):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * phase
            y[..., first], y[..., second] = z.real.contiguous(), z.imag.contiguous()
            return y

        if case["cache"] != "bf16":
            return {"q": rotated(s["q"]), "cache": None, "scale": None}
        cache = s["cache"].double()
        flat = cache.permute(0, 3, 1, 2, 4).reshape(-1, 2, kv, d).clone()
        keep = s["slots"] >= 0
        flat[s["slots"][keep], 0] = rotated(s["k"])[keep]
        flat[s["slots"][keep], 1] = s["v"].double()[keep]
        return {"q": rotated(s["q"]), "cache": flat.view(-1, page, 2, kv, d).permute(0, 2, 3, 1, 4).contiguous()}
    out = torch.zeros(rows, h, d, device=DEVICE, dtype=torch.float64)
    lse = torch.full((rows, h), -math.inf, device=DEVICE, dtype=torch.float64)
    lens = s["len"].tolist() if case["op"] == "decode" else None
    index = s["index"].tolist()
    for r in range(rows):
        at = torch.arange(lens[index[r]], device=DEVICE) if lens else s["ids"][r][s["ids"][r] >= 0].long()
        if at.numel() == 0:
            continue
        where = s["table"][index[r]].long()[at // page]
        x = s["cache"][where, :, :, at % page]  # [tokens, 2, kv heads, dim]
        if s["scale"] is None:
            x = x.double()
        else:
            x = x.view(torch.float8_e4m3fn).double() * s["scale"][where, :, :, at % page].double().unsqueeze(-1)
        score = torch.einsum("gid,tgd->git", s["q"][r].double().view(kv, h // kv, d), x[:, 0]) / math.sqrt(d)
        lse[r] = torch.logsumexp(score, -1).view(h)
        out[r] = torch.einsum("git,tgd->gid", torch.softmax(score, -1), x[:, 1]).reshape(h, d)
    return {"out": out, "lse": lse}
