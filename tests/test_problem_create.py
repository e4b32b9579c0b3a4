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
