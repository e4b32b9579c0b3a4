"""Creation of a problem and the cache entry points' refusals, in a process whose
CUDA runtime calls are the stand-ins of fake_cudart.c.  CPU only."""
import os
import subprocess
import sys

import pytest

from paged_varlen_flash_gb300 import build as ua_build

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

PRELUDE = """
import ctypes
import paged_varlen_flash_gb300 as ua
fake = ctypes.CDLL(None)
fake.fake_allocated.restype = ctypes.c_size_t

def create(**over):
    kw = dict(num_q_heads=8, num_kv_heads=2, head_size=128, block_size=16, num_blocks=64, max_num_seqs=4,
              max_blocks_per_seq=8, max_total_q=64, flags=ua.UA_FLAG_CAUSAL, scale=0.125)
    kw.update(over)
    return ua.ua_problem_create(**kw)

def status(**over):
    try:
        ua.ua_destroy(create(**over))
    except ua.UAError as e:
        return e.status
    return 0
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """Runs a script behind PRELUDE; a failed assertion in it fails the test."""
    ua_build.build()
    lib = str(tmp_path_factory.mktemp("fake") / "libfake_cudart.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", os.path.join(HERE, "fake_cudart.c"), "-o", lib], check=True)

    def go(script):
        r = subprocess.run([sys.executable, "-c", PRELUDE + script], cwd=ROOT, capture_output=True, text=True,
                           env=dict(os.environ, LD_PRELOAD=lib), timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr

    return go


def test_buffers_are_cleared_when_creation_returns(run):
    """No clearing is left in a stream: the first call may come on another one."""
    run("""
for kv in (ua.UA_DTYPE_BF16, ua.UA_DTYPE_FP4_E2M1):
    p = create(kv_dtype=kv, flags=ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    assert fake.fake_pending() == 0
    ua.ua_destroy(p)
""")


def test_sizes_past_64_bits_are_refused(run):
    """Workspaces whose byte counts wrap around are no small workspaces."""
    run("""
KW, FP4 = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS, ua.UA_DTYPE_FP4_E2M1
for tokens in (1 << 50, 1 << 52, (1 << 57) + 1, (1 << 62) + 1):
    assert status(max_total_q=tokens, flags=KW, num_q_heads=64, num_kv_heads=64, max_blocks_per_seq=512) == 4, tokens
    assert status(max_total_q=tokens, kv_dtype=FP4, num_q_heads=64, num_kv_heads=64) == 4, tokens
# Not so large: as before, the partials of a plain problem under their cap.
before = fake.fake_allocated()
assert status(max_total_q=1 << 62) == 0
assert (128 << 20) <= fake.fake_allocated() - before < (10 << 30)
before = fake.fake_allocated()
assert status(max_total_q=8, flags=KW) == 0
scores, work = 4 * 8 * 8 * 128, fake.fake_allocated() - before
assert 4 * 8 * 8 * 16 * 130 + scores < work < 4 * 8 * 8 * 16 * 130 + scores + (1 << 20)
""")


def test_misaligned_arrays_are_refused(run):
    """int32 and fp32 arrays off their 4-byte boundary; nothing is launched (a call
    that passes the checks ends in a CUDA error here)."""
    run("""
p = create(flags=ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS | ua.UA_FLAG_SINKS | ua.UA_FLAG_ALIBI,
           kv_dtype=ua.UA_DTYPE_FP4_E2M1)
A = 1 << 12                                   # an address that only the checks look at
flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_SINKS | ua.UA_FLAG_ALIBI

def forward(table=A, cu=A, used=A, sinks=A, alibi=A):
    return ua.ua_forward(p, A, A, A, table, cu, used, 2, 2, 1, 40, flags, sinks, alibi, A, stream=0)

def weights(table=A, cu=A, used=A, sinks=A, alibi=A, w_in=A, w_out=A):
    return ua.ua_forward_weights(p, A, A, A, table, cu, used, 2, 2, 1, 40, flags, sinks, alibi, w_in, w_out, 40, 1.0,
                                 A, stream=0)

def store(table=A, cu=A, used=A):
    return ua.ua_cache_store(p, A, A, 256, A, A, table, cu, used, 2, 2, 1, 40, stream=0)

def expand(table=A, used=A, begin=A, out=A):
    return ua.ua_cache_expand(p, A, A, table, used, begin, 2, 40, A, A, out, 8, 64, stream=0)

def evict(table=A, dst=A + 64, used=A, w_in=A, w_out=A, kept=A, used_out=A):
    return ua.ua_cache_evict(p, A, A, table, dst, used, 2, 40, w_in, w_out, 40, 10, 2, kept, used_out, stream=0)

for call in (forward, weights, store, expand, evict):
    assert call() == 3, (call.__name__, call())
    for name in call.__code__.co_varnames[:call.__code__.co_argcount]:
        for off in (1, 2, 3):
            assert call(**{name: A + off}) == 1, (call.__name__, name)
""")
