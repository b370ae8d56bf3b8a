"""The checked build runs the further GPU tests of the 8-bit cache green: values
far apart and not finite, every form over long prefixes, the largest tables,
steps with trees of other sizes."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

from tree_verification_jsv_b200 import build as jbuild

ROOT = Path(__file__).resolve().parents[1]

pytestmark = pytest.mark.gpu


def test_checked_build_runs_the_further_kv8_tests_clean():
    jbuild.build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_kv8_scales.py", "tests/test_gpu_kv8_nonfinite.py", "tests/test_gpu_kv8_forms.py",
                        "tests/test_gpu_kv8_limits.py", "tests/test_gpu_kv8_step_sizes.py", "-k", "not shared"],
                       cwd=ROOT, env=dict(os.environ, JSV_LIBRARY="checked"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
