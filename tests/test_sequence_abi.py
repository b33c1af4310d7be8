"""Refusals of the sequences' attention and of the page operators that need no GPU, the struct layouts of the binding, and the
plain forms of their tests against worked examples."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

import sparse_attention_top_expand_gb300 as smq
from sparse_attention_top_expand_gb300.csrc import build as libbuild

import pages_ref
import sequence_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return smq.load_library()


def test_struct_layouts_match_binding(tmp_path):
    fields = {"smq_seq_attention_args": smq.SMQSeqAttentionArgs, "smq_page_plan_desc": smq.SMQPagePlanDesc,
              "smq_page_plane": smq.SMQPagePlane, "smq_pages_resize_args": smq.SMQPagesResizeArgs,
              "smq_pages_fork_args": smq.SMQPagesForkArgs, "smq_cache_compact_args": smq.SMQCacheCompactArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "smq.h"', "int main(void) {"]
    for cname, cls in fields.items():
        lines.append(f'  printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    lines += ['  printf("planes %d\\n", SMQ_MAX_PLANES);', '  printf("nopages %d\\n", SMQ_ERR_NO_PAGES);']
    prog, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    prog.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["planes"]) == smq.SMQ_MAX_PLANES
    assert int(got["nopages"]) == smq.SMQ_ERR_NO_PAGES == pages_ref.NO_PAGES
    for cname, cls in fields.items():
        assert int(got[cname]) == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, f"{cname}.{f}"


def test_null_arguments_rejected(lib):
    n = ctypes.c_size_t()
    bad = smq.SMQ_ERR_INVALID_ARG
    assert lib.smq_seq_attention_workspace_size(None, ctypes.byref(n)) == bad
    assert lib.smq_page_plan_create(None, None) == bad
    assert lib.smq_page_workspace_size(None, ctypes.byref(n)) == bad
    assert lib.smq_page_workspace_init(None, None, 0, None) == bad
    for call in (lib.sparse_mqa_attention_window, lib.sparse_mqa_attention_tree, lib.sparse_mqa_pages_resize,
                 lib.sparse_mqa_pages_fork, lib.sparse_mqa_cache_compact):
        assert call(None, None, None) == bad


def test_status_words_have_names(lib):
    for code in (smq.SMQ_ERR_NO_PAGES, smq.SMQ_ERR_NO_PAGES | smq.SMQ_ERR_BOUNDS):
        assert b"free pages" in lib.smq_error_string(code)


def test_window_sets_by_hand():
    got = [s.tolist() for s in sequence_ref.window_sets(3, 6, 2, 1)]
    assert got == [[0, 2, 3], [0, 3, 4], [0, 4, 5]]
    assert [s.tolist() for s in sequence_ref.window_sets(3, 2, 5, 0)] == [[], [0], [0, 1]]


def test_tree_sets_by_hand():
    got = [s.tolist() for s in sequence_ref.tree_sets(3, 5, [{0}, {0, 1}, {0, 2, 9}])]
    assert got == [[0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 4]]
    assert sequence_ref.pack([{0, 31, 32}, set()], 2).tolist() == [[-2 ** 31 + 1, 1], [0, 0]]


def test_the_pool_by_hand():
    p = pages_ref.Pool(4, 6, 3, 3)
    p.planes = [np.arange(6 * 1 * 4).reshape(6, 1, 4)]
    assert p.resize([9, 4, 0]) == 0
    assert p.table.tolist() == [[0, 1, 2], [3, -1, -1], [-1, -1, -1]] and p.refs.tolist() == [1, 1, 1, 1, 0, 0]
    assert p.fork([0], [2], [6]) == 0
    assert p.table[2].tolist() == [0, 4, -1] and p.refs.tolist() == [2, 1, 1, 1, 1, 0]
    assert p.planes[0][4, 0].tolist() == [4, 5, 18, 19]
    assert p.compact([5], [[6, 8, -1]], rows=[0]) == 0
    assert p.planes[0][1, 0].tolist() == [4, 6, 8, 7]
    assert p.compact([1], [[2]], rows=[0]) == pages_ref.BOUNDS  # the place is in a page that two rows hold
    assert p.resize([0, 0, 12]) == 0  # row 2 wants one page, and page 5 was free before the call
    assert p.table[2].tolist() == [0, 4, 5] and p.refs.tolist() == [1, 0, 0, 0, 1, 1]
