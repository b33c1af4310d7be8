"""The drafting example runs, its pages add up, and where a window covers a context the window's result is the tree's root's."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache_dtype", ["bf16", "e4m3"])
def test_steps_of_drafted_decoding(cache_dtype):
    spec = importlib.util.spec_from_file_location("draft_tree_step", os.path.join(ROOT, "examples", "draft_tree_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    batch = example.Batch([700, 100, 64, 400], cache_dtype=cache_dtype)
    for _ in range(5):
        before = batch.lens.clone()
        out, local, accepted = batch.step()
        assert torch.equal(batch.lens, before + accepted) and bool((accepted >= 1).all())
        pages = (batch.lens + example.PAGE - 1) // example.PAGE
        held = batch.table >= 0
        assert torch.equal(held.sum(1), pages)
        counts = torch.zeros_like(batch.refs).index_add_(0, batch.table[held].long(), torch.ones_like(batch.table[held]))
        assert torch.equal(counts, batch.refs), "every page has as many holders as the table says"
        for r, n in enumerate(before.tolist()):
            if n + 1 <= example.WINDOW:  # the same tokens: sums in another order, results of 8 bits
                off = (out[r, 0].float() - local[r].float()).abs().max()
                assert off <= 2 ** -7 * local[r].float().abs().max(), (r, float(off))
    assert int((batch.refs > 1).sum()) == 700 // example.PAGE, "the two samples share the prompt's whole pages"
