"""A wait limit that any call may overrun: the kernel may give up at any of its waits, and must leave nothing in flight."""

import numpy as np
import pytest
import torch

import sparse_attention_top_expand_gb300 as smq

import attention_ref as ref
from test_attention_gpu import Rows

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("heads,kv_heads,dtype", [(64, 1, "bf16"), (16, 2, "bf16"), (64, 1, "e4m3"), (128, 1, "e4m3")])
def test_a_limit_of_a_nanosecond_ends_every_call(heads, kv_heads, dtype):
    rng = np.random.Generator(np.random.PCG64(31))
    lens = [900, 5, 640, 0]
    cache = ref.Cache(rng, kv_heads, 128, 64, dtype, lens)
    seqs = [i % 4 for i in range(152)]
    rows = Rows(rng, cache, heads, seqs)
    counts = [lens[s] for s in seqs]
    ke = torch.tensor(counts, dtype=torch.int32, device=DEV)
    rows.plan.set_wait_limit(1)
    for _ in range(5):
        status = rows.call(row_ke=ke)
        assert status in (0, smq.SMQ_ERR_TIMEOUT)
        if status == 0:
            rows.check([np.arange(n) for n in counts], rows=[0, 1, 150])
        smq.smq_attn_workspace_init(rows.plan, rows.dev["workspace"])
    rows.plan.set_wait_limit(2_000_000_000)
    assert rows.call(row_ke=ke) == 0
    rows.check([np.arange(n) for n in counts], rows=[0, 1, 2, 3, 77, 151])
