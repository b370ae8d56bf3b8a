"""The checked build (every computed global index compared with its buffer's
extent) runs the 8-bit cache's and the page pool's GPU tests green."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

from tree_verification_jsv_b200 import build as jbuild

ROOT = Path(__file__).resolve().parents[1]

pytestmark = pytest.mark.gpu


def test_checked_build_runs_the_kv8_and_pool_tests_clean():
    jbuild.build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_kv8.py", "tests/test_gpu_kv8_tiles.py", "tests/test_gpu_pages.py",
                        "tests/test_gpu_kv8_step.py"],
                       cwd=ROOT, env=dict(os.environ, JSV_LIBRARY="checked"), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
