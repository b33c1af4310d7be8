"""Inputs that a test chooses token by token for the attention operators, their plain 64-bit results, and how far a bf16
result of the kernel's arithmetic can be from them."""

import math

import numpy as np
import torch

import attention_ref as ref


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def put(cache, seq, positions, side, x, scales=None):
    """Keys (side 0) or values (side 1) of positions of a sequence of an attention_ref.Cache: x [tokens, kv heads, dim].
    With scales [tokens, kv heads], x holds E4M3 codes (uint8) instead."""
    p = np.asarray(positions, np.int64)
    page, off = cache.table[seq][p // cache.page].astype(np.int64), p % cache.page
    tp, to = torch.from_numpy(page), torch.from_numpy(off)
    if cache.dtype == "bf16":
        t = bf16(x)
        cache.data[tp, side, :, to] = t
        cache.values[page, side, :, off] = t.to(torch.float64).numpy()
        return
    if scales is None:
        x, scales = ref.quantise(x)
    cache.data[tp, side, :, to] = torch.from_numpy(np.ascontiguousarray(x))
    cache.scales[tp, side, :, to] = torch.from_numpy(np.ascontiguousarray(scales, np.float32))
    cache.values[page, side, :, off] = ref.e4m3_values(x) * np.asarray(scales, np.float64)[..., None]


def attend(q, k, v, scale):
    """q [H, D], k and v [tokens, KVH, D] in 64 bits: out and the mean of |v| under the softmax [H, D], lse and, of the
    tokens that have any weight, the largest sum of |q||k| in units of a score [H]."""
    h, d = q.shape
    group = h // k.shape[1]
    out, mean = np.zeros((h, d)), np.zeros((h, d))
    lse, size = np.zeros(h), np.zeros(h)
    for i in range(h):
        kk, vv = k[:, i // group], v[:, i // group]
        s = (kk @ q[i]) * scale
        m = s.max()
        p = np.exp(s - m)
        lse[i] = m + math.log(p.sum())
        p /= p.sum()
        out[i], mean[i] = p @ vv, p @ np.abs(vv)
        size[i] = (np.abs(kk[p > 2.0 ** -40]) @ np.abs(q[i])).max() * abs(scale)
    return out, mean, lse, size


def bound(out, mean, size, dim, tokens):
    """The largest error of a bf16 result, and of its lse.

    Scores: dim / 16 steps of the tensor core, each adding 16 exact products to the accumulator, 17 terms cut at 2^-24 of
    the largest at worst; then at most five roundings to 2^-24 (scales, maximum). A weight moves by exp of that, and by
    2^-21 of the exponential's own error; out moves with the weights and with their sum.
    Weights: hi is cut to 8 bits, lo holds what is left to 8 bits more: 2^-15 of each.
    Values: 8 steps as above for each tile of 128 tokens, and 2^-20 of sums and joins.
    The result is then rounded to the nearest of 8 bits: half a step."""
    score = size * (dim / 16 * 17 + 5) * 2.0 ** -24
    moved = (np.expm1(score) + 2.0 ** -21)[:, None]
    off = (np.abs(out) + mean) * moved + mean * (2.0 ** -15 + 8 * math.ceil(tokens / 128) * 17 * 2.0 ** -24 + 2.0 ** -20)
    top = np.maximum(np.abs(out) + off, 2.0 ** -126)
    return off + 2.0 ** (np.floor(np.log2(top)) - 8), score + 2.0 ** -20


def check(got, lse, q, k, v, scale, where="", absolute=0.0):
    """A row's result [H, D] and lse [H] against the plain form, within bound() and `absolute`."""
    out, mean, want_lse, size = attend(q, k, v, scale)
    off, lse_off = bound(out, mean, size, q.shape[1], len(k))
    got, lse = got.to(torch.float64).cpu().numpy(), lse.to(torch.float64).cpu().numpy()
    assert np.isfinite(got).all(), f"{where}: not finite"
    over = np.abs(got - out) - off - absolute
    assert (over <= 0).all(), (f"{where}: {(over > 0).sum()} of {over.size} over the bound, by {over.max():.3g}; off by "
                               f"{np.linalg.norm(got - out) / np.linalg.norm(out):.3g} of the norm")
    over = np.abs(lse - want_lse) - lse_off - 2.0 ** -22 * np.abs(want_lse)
    assert (over <= 0).all(), f"{where}: lse over its bound by {over.max():.3g}"
