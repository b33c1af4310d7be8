"""The bound of the sequences' attention in the attention plan, through the C ABI, without a GPU."""

import ctypes

import pytest

import sparse_attention_top_expand_gb300 as smq
from sparse_attention_top_expand_gb300.csrc import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return smq.load_library()


def _create(lib, size=None, **kw):
    d = dict(num_heads=64, num_kv_heads=8, head_dim=128, page_size=64, cache_type=0, max_rows=64, device=0, softmax_scale=0.0,
             max_sequence_rows=0)
    d.update(kw)
    h = ctypes.c_void_p()
    rc = lib.smq_attn_plan_create(ctypes.byref(smq.SMQAttnPlanDesc(size or ctypes.sizeof(smq.SMQAttnPlanDesc), *d.values())),
                                  ctypes.byref(h))
    if h.value:
        lib.smq_attn_plan_destroy(h)
    return rc


PASSES = (smq.SMQ_OK, smq.SMQ_ERR_CUDA)  # without a GPU the check of the device is the next one


@pytest.mark.parametrize("rows,code", [(-1, smq.SMQ_ERR_INVALID_ARG), (2 ** 20 + 1, smq.SMQ_ERR_UNSUPPORTED)])
def test_bounds_that_are_refused(lib, rows, code):
    assert _create(lib, max_sequence_rows=rows) == code


@pytest.mark.parametrize("rows", [0, 1, 8193, 2 ** 20])
def test_bounds_that_pass(lib, rows):
    assert _create(lib, max_sequence_rows=rows) in PASSES


def test_a_description_without_the_bound_is_taken(lib):
    old = smq.SMQAttnPlanDesc.max_sequence_rows.offset
    assert _create(lib, size=old, max_sequence_rows=-5) in PASSES  # past its end, not read
    assert _create(lib, size=old - 1) == smq.SMQ_ERR_INVALID_ARG


def test_numbers_past_32_bits_are_refused(lib):
    """2^32 + 64 is not 64."""
    wide = 2 ** 32 + 64
    for make in (lambda: smq.AttentionPlan(4, 2, 64, 16, max_rows=wide, device=0),
                 lambda: smq.PagePlan(wide, 10, 4, 4, device=0), lambda: smq.PagePlan(16, 10, wide, 4, device=0),
                 lambda: smq.PagePlan(16, 10, 4, wide, device=0)):
        with pytest.raises(ValueError, match="32 bits"):
            make()
