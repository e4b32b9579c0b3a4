"""Refusals of the step calls that a launch must not be needed for, in a process without a
GPU, and frequencies of long trained contexts.  CPU only."""
import math

import pytest

import paged_varlen_flash_gb300 as ua
from tests.test_problem_create import run  # noqa: F401

TREE = """
CAUSAL = ua.UA_FLAG_CAUSAL
A = 1 << 12                                   # an address that only the checks look at

def tree(p, max_q=4, max_k=40):
    return ua.ua_forward_tree(p, A, A, A, A, A, A, 2, 4, max_q, max_k, A, 1, None, CAUSAL, None, None, A, stream=0)
"""


def test_trees_of_more_kv_heads_than_a_grid_has(run):
    """Whatever the cache holds: no other kernel, which would not know the mask, takes the call."""
    run(TREE + """
for kind in (ua.UA_DTYPE_BF16, ua.UA_DTYPE_FP8_E4M3, ua.UA_DTYPE_FP4_E2M1):
    for heads, want in ((65536, 2), (65535, 3)):         # 3: the launch, without a GPU
        p = create(kv_dtype=kind, num_q_heads=heads, num_kv_heads=heads, max_total_q=4)
        assert tree(p) == want, (kind, heads, tree(p))
        ua.ua_destroy(p)
""")


def test_trees_over_more_keys_than_are_served(run):
    run(TREE + """
for kind in (ua.UA_DTYPE_BF16, ua.UA_DTYPE_FP8_E4M3, ua.UA_DTYPE_FP4_E2M1):
    p = create(kv_dtype=kind, max_blocks_per_seq=(1 << 26) + 1, max_total_q=4)
    assert tree(p, max_k=(1 << 30) + 1) == 2 and tree(p, max_k=1 << 30) == 3, kind
    ua.ua_destroy(p)
""")


@pytest.mark.parametrize("rotated,base,trained,factor", [(128, 10000.0, 131072, 4.0), (128, 10000.0, 131072, 8.0),
                                                         (64, 500000.0, 1 << 25, 2.0), (16, 100.0, 4096, 8.0)])
def test_yarn_ramps_that_end_behind_the_last_pair(rotated, base, trained, factor):
    """Where even the last pair makes more than ``low`` turns, it keeps a part of its frequency."""
    n, low, high = rotated // 2, 1.0, 32.0
    plain = ua.rope_frequencies(rotated, base)[0]
    yarn, _ = ua.rope_frequencies(rotated, base, "yarn", factor, trained, low, high)
    number = lambda turns: n * math.log(trained / (2 * math.pi * turns), base)  # noqa: E731
    first, end = math.floor(number(high)), min(math.ceil(number(low)), rotated - 1)
    assert trained * plain[-1] / (2 * math.pi) > low and end >= n
    for i, (f, y) in enumerate(zip(plain, yarn)):
        keep = min(1.0, 1 - (i - first) / (end - first))
        assert math.isclose(y, f * (keep + (1 - keep) / factor), rel_tol=1e-9), i
    assert yarn[-1] > plain[-1] / factor * 1.001
