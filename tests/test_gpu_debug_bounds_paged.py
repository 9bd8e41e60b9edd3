"""The bounds-checking debug build (-DDSA_DEBUG_BOUNDS=1) and the paged cache:
its kernels check table entries, list entries, cache rows, parts and outputs
before they use them.  A child process loads that build (DSA_LIB) and runs the
four calls on edge shapes; none may report."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_bounds_build_runs_the_paged_calls_clean():
    from sparse_attention_token_index_b200 import build as B
    env = dict(os.environ, DSA_LIB=B.build(debug_bounds=True))
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_bounds_paged.py")], env=env, cwd=os.path.dirname(HERE),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "debug-bounds cases ok" in r.stdout
