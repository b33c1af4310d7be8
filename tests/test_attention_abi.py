"""Refusals of the attention operators that need no GPU: the plan's geometry and null arguments through the C ABI, and
the struct layouts of the binding."""

import ctypes
import os
import subprocess

import pytest

import sparse_attention_top_expand_gb300 as smq
from sparse_attention_top_expand_gb300.csrc import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return smq.load_library()


def test_struct_layouts_match_binding(tmp_path):
    fields = {"smq_attn_plan_desc": smq.SMQAttnPlanDesc, "smq_append_args": smq.SMQAppendArgs,
              "smq_attention_args": smq.SMQAttentionArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "smq.h"', "int main(void) {"]
    for cname, cls in fields.items():
        lines.append(f'  printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    prog, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    prog.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for cname, cls in fields.items():
        assert int(got[cname]) == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, f"{cname}.{f}"


def _create(lib, **kw):
    d = dict(num_heads=64, num_kv_heads=8, head_dim=128, page_size=64, cache_type=0, max_rows=64, device=0, softmax_scale=0.0)
    d.update(kw)
    size = d.pop("struct_size", ctypes.sizeof(smq.SMQAttnPlanDesc))
    h = ctypes.c_void_p()
    rc = lib.smq_attn_plan_create(ctypes.byref(smq.SMQAttnPlanDesc(size, *d.values())), ctypes.byref(h))
    return rc, h


@pytest.mark.parametrize("bad,code", [
    (dict(num_heads=0), smq.SMQ_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), smq.SMQ_ERR_INVALID_ARG),
    (dict(num_heads=12), smq.SMQ_ERR_INVALID_ARG),          # not a multiple of the kv heads
    (dict(num_heads=129, num_kv_heads=1), smq.SMQ_ERR_UNSUPPORTED),
    (dict(num_heads=2048, num_kv_heads=64), smq.SMQ_ERR_UNSUPPORTED),
    (dict(num_heads=256, num_kv_heads=256), smq.SMQ_ERR_UNSUPPORTED),
    (dict(head_dim=96), smq.SMQ_ERR_UNSUPPORTED),
    (dict(page_size=0), smq.SMQ_ERR_INVALID_ARG),
    (dict(page_size=65537), smq.SMQ_ERR_UNSUPPORTED),
    (dict(cache_type=2), smq.SMQ_ERR_INVALID_ARG),
    (dict(max_rows=0), smq.SMQ_ERR_INVALID_ARG),
    (dict(max_rows=8193), smq.SMQ_ERR_UNSUPPORTED),
    (dict(device=-1), smq.SMQ_ERR_INVALID_ARG),
    (dict(softmax_scale=float("nan")), smq.SMQ_ERR_INVALID_ARG),
    (dict(softmax_scale=float("inf")), smq.SMQ_ERR_INVALID_ARG),
    (dict(struct_size=8), smq.SMQ_ERR_INVALID_ARG),
])
def test_plan_create_rejects_bad_geometry(lib, bad, code):
    rc, h = _create(lib, **bad)
    assert rc == code and not h.value


def test_valid_geometry_reaches_the_device_check(lib):
    rc, h = _create(lib)
    assert rc in (smq.SMQ_OK, smq.SMQ_ERR_CUDA, smq.SMQ_ERR_UNSUPPORTED)
    if rc == smq.SMQ_OK:
        lib.smq_attn_plan_destroy(h)


def test_null_arguments_rejected(lib):
    n = ctypes.c_size_t()
    bad = smq.SMQ_ERR_INVALID_ARG
    assert lib.smq_attn_plan_create(None, None) == bad
    assert lib.smq_attn_workspace_size(None, ctypes.byref(n)) == bad
    assert lib.smq_attn_workspace_init(None, None, 0, None) == bad
    assert lib.smq_attn_plan_set_wait_limit(None, 1) == bad
    assert lib.smq_attn_plan_inject_stall(None, 0) == bad
    for call in (lib.sparse_mqa_append_kv, lib.sparse_mqa_attention_decode, lib.sparse_mqa_attention_selected):
        assert call(None, None, None) == bad
