"""The bound that the attention tests use, against a model of the kernel's arithmetic on the CPU: it holds for weights of
two bf16 numbers, and not where the second is lost or holds another's rest."""

import numpy as np
import pytest
import torch

import attention_bounds as ab


def _model(q, k, v, scale, parts):
    """Scores, exponentials and sums in fp32, weights cut to `parts`, values summed in 64 bits, bf16 at the end."""
    s = (q.astype(np.float32) @ k[:, 0].astype(np.float32).T) * np.float32(scale)
    p = np.exp(s - s.max(1, keepdims=True)).astype(np.float32)
    hi = (p.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    lo = torch.from_numpy(p - hi).to(torch.bfloat16).float().numpy()
    weights = {"both": hi + lo, "hi": hi, "wrong lo": hi + np.roll(lo, 1, 1)}[parts].astype(np.float64)
    out = torch.from_numpy(weights @ v[:, 0] / p.sum(1, keepdims=True, dtype=np.float64)).to(torch.bfloat16)
    return out, torch.from_numpy(s.max(1) + np.log(p.sum(1)))


@pytest.mark.parametrize("n", [1, 2, 127, 300, 1000, 5000])
@pytest.mark.parametrize("parts", ["both", "hi", "wrong lo"])
def test_the_bound_tells_a_lost_half(n, parts):
    rng = np.random.Generator(np.random.PCG64(n))
    q = ab.bf16(rng.standard_normal((16, 128)) * 1.5).to(torch.float64).numpy()
    k, v = (ab.bf16(rng.standard_normal((n, 1, 128))).to(torch.float64).numpy() for _ in range(2))
    out, lse = _model(q, k, v, 128 ** -0.5, parts)
    if parts == "both" or n == 1:  # a single weight is 1, without a low half
        ab.check(out, lse, q, k, v, 128 ** -0.5)
    elif n <= 1000:  # over thousands of tokens the values cancel, and the bound on their sum hides it
        with pytest.raises(AssertionError):
            ab.check(out, lse, q, k, v, 128 ** -0.5)
