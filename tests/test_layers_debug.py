"""A subset of the layers' tests under the bounds-checked build: every direct
global access of their kernels is checked against its buffer there, and each test
asserts a clear status word (see test_debug_build.py)."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SUBSET = "bf16 or f32 or many or mlp or cuda_cores"


def test_layers_under_the_bounds_checked_library():
    from rank_structured_matmul_b200.build import build
    build(debug=True)  # incremental: rebuilt only when a source is newer
    env = dict(os.environ, DYRA_DEBUG_LIB="1")
    out = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_layers.py"),
                          "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider", "-k", SUBSET],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (out.stdout + out.stderr)[-3000:]
    assert out.returncode == 0, tail
    assert " passed" in out.stdout and "error" not in out.stdout.lower().split("passed")[-1], tail
