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
