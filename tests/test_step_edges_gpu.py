"""Step calls at the edges of what their documentation allows: batches without rows,
positions out of range, results that a call allocates, budgets that are met, far angles,
tables of 16384 sequences, random rotary stores.  Tolerances: tests/test_step_ops_gpu.py
where nothing else is said."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests import step_ref as S
from tests.test_step_ops_gpu import Planned, Trees, _built, check_rotated, i32, same  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- no rows allowed
@pytest.mark.parametrize("kind,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp8", 128), ("fp4", 64), ("fp4", 128),
                                    ("fp4", 256)])
def test_trees_of_a_batch_without_rows(kind, d):
    """max_seqlen_q = 0 with padding tokens: empty sequences are served, others reported."""
    bt = Trees(2000, 8, 2, d, 16, (2, 3), (40, 20), kind=kind).device()
    p = bt.problem()
    mask = torch.from_numpy(bt.mask.view(np.int32)).cuda()
    out = torch.full_like(bt.d_q, 7.0)

    def call(cu, sk, most):
        p.forward_tree(bt.d_q, bt.d_k, bt.d_v, bt.d_table, cu, sk, 2, 5, 0, most, ua.UA_FLAG_CAUSAL, mask, out=out)

    for sk, most in ((bt.d_sk, 40), (i32([0, 0]), 40), (i32([0, 0]), 0)):
        call(i32([0, 0, 0]), sk, most)
        assert p.check_device_error() == 0 and bool((out == 7).all())
    call(bt.d_cu, bt.d_sk, 40)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS and bool((out == 0).all())
