"""Refusals of the step calls that a launch must not be needed for: the library's, in a
process without a GPU, and the binding's.  CPU only."""
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
