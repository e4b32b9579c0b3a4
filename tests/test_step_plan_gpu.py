"""Step plans on the GPU that are short of blocks and of places, give back what they should
not hold, or are of very many sequences, against the lists of tests/step_ref.py.  Exact."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import step_ref as S
from tests.test_step_ops_gpu import Planned, _built, i32, same  # noqa: F401

pytestmark = pytest.mark.gpu

# ---------------------------------------------------------------- the plan's budgets
def served(held, ctx, new, b, pool, cap):
    """Who gets tokens: in order, blocks from the pool counted over all that ask for some,
    places over all that the pool serves."""
    asked = tokens = err = 0
    out = []
    for h, c, k in zip(held, ctx, new):
        more = max(0, -(-(c + k) // b) - h)
        asked += more
        if more and asked > pool:
            out.append(0)
            continue
        tokens += k
        err |= S.BOUNDS if k and tokens > cap else 0
        out.append(k if tokens <= cap else 0)
    return out, err


def test_tokens_that_the_pool_refuses_need_no_places():
    st = Planned(2200, 4, 16, pool=0, ctx=[16, 5, 5, 7], spare=0)
    out = st.outputs(7)
    st.problem.plan_step(st.table, st.held, st.pool, st.left, i32(st.ctx), i32([10, 3, 4, 0]), 4, 7, **out)
    assert st.problem.check_device_error() == 0
    same(out["granted"], [0, 3, 4, 0])
    same(out["cu_seqlens_q"], [0, 0, 3, 7, 7])
    same(out["seqused_k"], [16, 8, 9, 7])
    same(out["positions"], [5, 6, 7, 5, 6, 7, 8])


@pytest.mark.parametrize("n,seed", [(3, 0), (40, 1), (256, 2), (257, 3), (1500, 4), (5000, 5)])
def test_plans_short_of_blocks_and_places(n, seed):
    g = np.random.default_rng(2300 + seed)
    b, width = 16, 8
    for share in (0.3, 0.7, 0.9):
        ctx = [int(x) for x in g.integers(0, 60, n)]
        new = [int(x) for x in g.integers(0, 40, n)]
        held = [-(-c // b) for c in ctx]
        want_blocks = sum(max(0, -(-(c + k) // b) - h) for c, k, h in zip(ctx, new, held))
        pool, cap = int(share * want_blocks), max(1, int(g.uniform(0.2, 1.0) * sum(new)))
        st = Planned(2400 + seed, n, b, width=width, num_blocks=8 * n + 64, pool=pool, ctx=ctx, spare=0)
        granted, err = served(held, ctx, new, b, pool, cap)
        out = st.outputs(cap)
        st.problem.plan_step(st.table, st.held, st.pool, st.left, i32(ctx), i32(new), n, cap, **out)
        assert st.problem.check_device_error() == err
        same(out["granted"], granted)
        # What is given out is what a step of these tokens alone gets.
        want, none = st.ref.plan(ctx, granted, cap)
        assert none == 0
        st.check(want, out, cap, 0)


@pytest.mark.parametrize("n", [3920, 3924, 3925, 4100, 16384])
def test_plans_whose_sums_need_more_shared_memory(n):
    """12 bytes a sequence: up to the largest number of them."""
    g = np.random.default_rng(n)
    st = Planned(2500 + n, n, 16, width=4, num_blocks=5 * n, pool=n // 2, ctx=[int(x) for x in g.integers(0, 30, n)])
    for tree in (False, True):
        new = [int(x) for x in g.integers(0, 5, n)]
        st.step(new, sum(new) + 3, [S.grow(g, k) for k in new] if tree else None, 1 if tree else 0)
        st.step([0] * n, 1)


@pytest.mark.parametrize("bad", [-1, 200, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("taken", [False, True])
def test_bad_ids_that_are_given_back_are_reported(bad, taken):
    """When they go to the pool, not only when somebody takes them from there again."""
    st = Planned(2600, 4, 16, pool=5, ctx=[40, 16, 33, 0], spare=0)
    st.ref.table[2][1] = bad
    st.upload()
    want = [st.ref.table[2][0], bad, st.ref.table[2][2]]
    new = [0, 0, 0, 16 * 2 if taken else 0]
    out = st.outputs(40)
    st.problem.plan_step(st.table, st.held, st.pool, st.left, i32([40, 16, 0, 0]), i32(new), 4, 40, **out)
    assert st.problem.check_device_error() == S.BLOCK_ID
    same(st.held, [3, 1, 0, 2 if taken else 0])
    same(st.left, [6 if taken else 8])
    # The first returned block lies on top; the last one below the others.
    if taken:
        same(st.table[3, :2], want[:2])
        same(out["slots"][:32], [want[0] * 16 + i for i in range(16)] + [-1] * 16)
        same(st.pool[:6], st.ref.pool + want[2:])
    else:
        same(st.pool[:8], st.ref.pool + want[::-1])
