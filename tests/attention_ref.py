"""Plain 64-bit forms of the attention operators, on the CPU, and the inputs of their tests. No code shared with the
library: positions are looked up one by one, products and exponentials are numpy's."""

import math

import numpy as np
import torch


def quantise(x):
    """float32 [..., D] to E4M3 codes (uint8) and scale = amax / 448 (1 for zeros), both divisions in float32."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(-1)
    scale = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
    q = torch.from_numpy((x / scale[..., None]).astype(np.float32)).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).numpy(), scale


def e4m3_values(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def rotate(x, cos, sin, interleaved):
    """x [T, heads, D] float32, cos and sin [T, pairs] float32; every product and sum rounded to float32."""
    x = np.asarray(x, np.float32)
    n = cos.shape[1]
    out = x.copy()
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = x[..., first], x[..., second]
    c, s = cos[:, None, :].astype(np.float32), sin[:, None, :].astype(np.float32)
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out


class Cache:
    """A paged cache of random keys and values, K and V views of one allocation; what no sequence owns is poison:
    NaN in a bf16 cache, E4M3 NaN codes and NaN scales in an 8-bit one."""

    def __init__(self, rng, kv_heads, dim, page, dtype, lens, spare=3):
        self.kv_heads, self.dim, self.page, self.dtype = kv_heads, dim, page, dtype
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        width = max(1, max(need))
        self.table = np.full((len(lens), width), order[-1], np.int32)
        values = rng.standard_normal((self.pages, 2, kv_heads, page, dim)).astype(np.float32)
        owned = np.zeros((self.pages, page), bool)
        at = 0
        for s, n in enumerate(lens):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for p in range(n):
                owned[self.table[s, p // page], p % page] = True
        poison = ~owned[:, None, None, :]
        if dtype == "bf16":
            t = torch.from_numpy(values).to(torch.bfloat16)
            self.values = t.to(torch.float64).numpy()
            t[torch.from_numpy(np.broadcast_to(poison, t.shape[:4]).copy())] = float("nan")
            self.data, self.scales = t, None
        else:
            codes, scale = quantise(values * np.exp(rng.standard_normal(values.shape[:4] + (1,))).astype(np.float32))
            self.values = e4m3_values(codes) * scale[..., None].astype(np.float64)
            codes[np.broadcast_to(poison, codes.shape[:4])] = 0x7F
            scale[np.broadcast_to(poison, scale.shape)] = np.nan
            self.data, self.scales = torch.from_numpy(codes), torch.from_numpy(scale)

    def to(self, device):
        d = self.data.to(device)
        s = None if self.scales is None else self.scales.to(device)
        return dict(k_cache=d[:, 0], v_cache=d[:, 1], k_scales=None if s is None else s[:, 0],
                    v_scales=None if s is None else s[:, 1])

    def tokens(self, seq, positions):
        """Keys and values [tokens, kv heads, dim] in 64 bits."""
        p = np.asarray(positions, np.int64)
        page = self.table[seq][p // self.page]
        both = self.values[page, :, :, p % self.page]
        return both[:, 0], both[:, 1]


def attend(q, k, v, scale):
    """q [H, D], k and v [tokens, KVH, D] in 64 bits: out [H, D], lse [H], and for the tolerance the mean of |v| under
    the softmax [H, D], the largest weight [H] and the sum of |v| [H, D]."""
    h, d = q.shape
    kvh = k.shape[1]
    out, lse = np.zeros((h, d)), np.full(h, -math.inf)
    mean, top, total = np.zeros((h, d)), np.zeros(h), np.zeros((h, d))
    if len(k):
        for i in range(h):
            g = i // (h // kvh)
            s = (k[:, g] @ q[i]) * scale
            m = s.max()
            p = np.exp(s - m)
            lse[i] = m + math.log(p.sum())
            p /= p.sum()
            out[i] = p @ v[:, g]
            mean[i] = p @ np.abs(v[:, g])
            top[i] = p.max()
            total[i] = np.abs(v[:, g]).sum(0)
    return out, lse, mean, top, total


def tolerance(out, mean, top, total, dtype):
    """The largest error of a bf16 result. Rounding the result: half a step, 2^-9 of it. Rounding the weights: 2^-9 of
    each in bf16; 2^-8 in two E4M3 numbers of 4 bits each, or half of the smallest step 2^-9 where the weight, held
    as 256 at its maximum, is tiny: 2^-18 of the largest weight. Scores: fp32 sums of at most 128 products, and
    queries held to 2^-19 of their amax over an 8-bit cache, move a weight by at most 5e-4 of itself."""
    weights = 2.0 ** -9 * mean if dtype == "bf16" else 2.0 ** -8 * mean + 2.0 ** -18 * top[..., None] * total
    return 2.0 ** -9 * np.abs(out) + weights + 5e-4 * (np.abs(out) + mean) + 1e-12
