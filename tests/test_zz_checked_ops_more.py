"""The checked build (device bounds checks compiled in) runs the operators' other
tests in a child process: norms over many rows, the tail class with next to no
mass, small temperatures, every number of top alternatives, single rows, tensors
from anywhere in memory.  Collected last (zz) because it builds a second
library."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operators_under_checked_build():
    from float8_mixed_precision_gb300 import build
    env = dict(os.environ, F8_LIBRARY=build.build(checked=True))
    tests = [f"tests/test_gpu_{n}.py" for n in ("norm_rows", "tail_mass", "entropy_gradient", "top_limits", "one_row",
                                                "nn_offsets", "distill_values", "streams")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *tests],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m is not None and int(m.group(1)) >= 180, tail
