"""Failure and refusal of the attention calls on the GPU, without a fault: a withheld hand-off with a short wait limit
runs a pipeline wait out, and arguments that do not fit are refused before anything is enqueued."""

import ctypes
import time

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_ref as ref
from test_attention_gpu import Rows

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("heads,kv_heads,dtype,tile", [(64, 1, "bf16", 0), (16, 2, "bf16", 2), (64, 1, "e4m3", 1)])
def test_a_withheld_tile_times_out_and_the_next_call_is_right(heads, kv_heads, dtype, tile):
    rng = np.random.Generator(np.random.PCG64(3))
    lens = [700] * 152  # several tiles for the first CTA
    cache = ref.Cache(rng, kv_heads, 128, 64, dtype, lens[:4])
    rows = Rows(rng, cache, heads, [i % 4 for i in range(152)])
    ke = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rows.plan.set_wait_limit(2_000_000)
    rows.plan.inject_stall(tile)
    t0 = time.perf_counter()
    assert rows.call(row_ke=ke) & smq.SMQ_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    rows.plan.inject_stall(-1)
    rows.plan.set_wait_limit(2_000_000_000)
    smq.smq_attn_workspace_init(rows.plan, rows.dev["workspace"])
    assert rows.call(row_ke=ke) == 0
    rows.check([np.arange(n) for n in lens], rows=[0, 77, 151])


def _tensors(dtype="bf16", rows=3):
    kind = torch.bfloat16 if dtype == "bf16" else torch.uint8
    data = torch.zeros(4, 2, 2, 16, 64, device=DEV, dtype=kind)
    scales = None if dtype == "bf16" else torch.ones(4, 2, 2, 16, device=DEV)
    plan = smq.AttentionPlan(8, 2, 64, 16, max_rows=4, cache_dtype=dtype)
    q = torch.zeros(rows, 8, 64, device=DEV, dtype=torch.bfloat16)
    args = dict(k_cache=data[:, 0], v_cache=data[:, 1], k_scales=None if scales is None else scales[:, 0],
                v_scales=None if scales is None else scales[:, 1], block_table=torch.zeros(4, 4, dtype=torch.int32, device=DEV),
                row_indices=None, out=torch.empty_like(q), workspace=plan.workspace())
    return plan, q, args


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.float32), TypeError),
    (dict(out="shape"), ValueError),
    (dict(k_cache="dtype"), TypeError),
    (dict(k_cache="inner"), ValueError),
    (dict(v_cache="pages"), ValueError),
    (dict(k_scales="extra"), ValueError),
    (dict(row_ke="shape"), ValueError),
    (dict(row_ke="cpu"), ValueError),
    (dict(row_ke=None), ValueError),
    (dict(token_ids="both"), ValueError),
    (dict(block_table="short"), ValueError),
])
def test_the_binding_refuses_what_does_not_fit(change, error):
    plan, q, args = _tensors()
    args["row_ke"] = _i32(3)
    (name, what), = change.items()
    if name == "q":
        q = q.to(what)
    elif name == "out":
        args["out"] = args["out"][:2]
    elif what == "dtype":
        args[name] = args[name].float()
    elif what == "inner":
        args[name] = args[name].transpose(1, 2)
    elif what == "pages":
        args[name] = args[name][:3]
    elif what == "extra":
        args[name] = torch.ones(4, 2, 16, device=DEV)
    elif what == "cpu":
        args[name] = args[name].cpu()
    elif what == "both":
        args[name] = _i32(3, 5)
    elif what == "short":
        args[name] = args[name][:2]
    else:
        args[name] = what if what is None else _i32(2)
    with pytest.raises(error):
        smq.AttentionCall(plan, q, **args)


@pytest.mark.parametrize("field,value,code", [
    ("rows", -1, smq.SMQ_ERR_INVALID_ARG), ("rows", 5, smq.SMQ_ERR_INVALID_ARG), ("q", None, smq.SMQ_ERR_INVALID_ARG),
    ("q_stride", 8 * 64 + 4, smq.SMQ_ERR_INVALID_ARG), ("q_stride", 64, smq.SMQ_ERR_INVALID_ARG),
    ("k_cache", None, smq.SMQ_ERR_INVALID_ARG), ("num_pages", 0, smq.SMQ_ERR_INVALID_ARG),
    ("page_stride", 2 * 16 * 64 - 16, smq.SMQ_ERR_INVALID_ARG), ("page_stride", 4 * 16 * 64 + 8, smq.SMQ_ERR_INVALID_ARG),
    ("block_table", None, smq.SMQ_ERR_INVALID_ARG), ("bt_stride", 0, smq.SMQ_ERR_INVALID_ARG),
    ("row_ke", None, smq.SMQ_ERR_INVALID_ARG), ("out", None, smq.SMQ_ERR_INVALID_ARG),
    ("workspace", None, smq.SMQ_ERR_INVALID_ARG), ("workspace_bytes", 256, smq.SMQ_ERR_WORKSPACE_TOO_SMALL),
    ("struct_size", 16, smq.SMQ_ERR_INVALID_ARG),
])
def test_the_library_refuses_bad_attention_arguments(field, value, code):
    plan, q, args = _tensors()
    call = smq.AttentionCall(plan, q, row_ke=_i32(3), **args)
    setattr(call.args, field, value)
    with pytest.raises(smq.SMQError) as e:
        call()
    assert e.value.code == code
    assert smq.smq_get_status(args["workspace"]) == 0


@pytest.mark.parametrize("field,value,code", [
    ("num_ids", 0, smq.SMQ_ERR_INVALID_ARG), ("num_ids", (1 << 20) + 1, smq.SMQ_ERR_INVALID_ARG),
    ("ids_ld", 4, smq.SMQ_ERR_INVALID_ARG), ("token_ids", None, smq.SMQ_ERR_INVALID_ARG),
])
def test_the_library_refuses_bad_id_lists(field, value, code):
    plan, q, args = _tensors()
    call = smq.AttentionCall(plan, q, token_ids=_i32(3, 5), **args)
    setattr(call.args, field, value)
    with pytest.raises(smq.SMQError) as e:
        call()
    assert e.value.code == code


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("field,value", [
    ("rows", 5), ("k", None), ("v_stride", 12), ("q_out", None), ("rot_dim", 24), ("rot_dim", 80), ("positions", None),
    ("cos_sin", None), ("num_positions", 0), ("slot_mapping", None), ("v_cache", None), ("k_scales", "other"),
])
def test_the_library_refuses_bad_append_arguments(dtype, field, value):
    plan, q, args = _tensors(dtype)
    kv = torch.zeros(3, 2, 64, device=DEV, dtype=torch.bfloat16)
    at = torch.zeros(3, dtype=torch.int64, device=DEV)
    call = smq.AppendCall(plan, q, kv, kv, at, torch.zeros(9, 32, device=DEV), at, args["k_cache"], args["v_cache"],
                          args["workspace"], q_out=args["out"], k_scales=args["k_scales"], v_scales=args["v_scales"])
    if value == "other":  # scales where there are none, none where there are
        value = kv.data_ptr() if dtype == "bf16" else None
    setattr(call.args, field, value)
    with pytest.raises(smq.SMQError) as e:
        call()
    assert e.value.code == smq.SMQ_ERR_INVALID_ARG


def test_a_plan_of_another_device_is_refused():
    plan, q, args = _tensors()
    call = smq.AttentionCall(plan, q, row_ke=_i32(3), **args)
    assert call.args.struct_size == ctypes.sizeof(smq.SMQAttentionArgs)
    with pytest.raises(smq.SMQError):
        smq.AttentionPlan(8, 2, 64, 16, max_rows=4, device=torch.cuda.device_count())
