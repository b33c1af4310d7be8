"""The decode-step example: where the indexer's selection covers a context, attention over the selected tokens is
attention over the whole context."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache_dtype", ["bf16", "e4m3"])
def test_selected_tokens_that_cover_the_context(cache_dtype):
    spec = importlib.util.spec_from_file_location("sparse_decode_step", os.path.join(ROOT, "examples", "sparse_decode_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    step = example.Step([0, 1, 300, 1800, 6000], longest=6100, cache_dtype=cache_dtype)
    for _ in range(2):
        out, whole, ids = step.run()
    lens = step.lens.tolist()
    assert (ids >= 0).sum(1).tolist() == [min(n, example.TOPK) for n in lens]
    for r, n in enumerate(lens):
        if n <= example.TOPK:
            assert sorted(ids[r][:n].tolist()) == list(range(n))
            # the same tokens in another order: sums round differently, results to bf16 (8 bits)
            off = (out[r].float() - whole[r].float()).abs().max()
            assert off <= 2 ** -7 * whole[r].float().abs().max(), (r, float(off))
        else:
            assert not torch.equal(out[r], whole[r])
