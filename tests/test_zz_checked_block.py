"""The checked build (device bounds checks compiled in) runs the tests of the GEMM
with epilogue, the activations' backward pass, rotary positions, the residual norm
and their modules in a child process: indexed global accesses of their kernels are
tested against their buffers first, and the tests assert a clean device status, so an
index outside its buffer fails the run.  Tests past 2^31 elements stay out, to keep
the run short.  Collected last (zz) because it builds a second library."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_operators_under_checked_build():
    from float8_mixed_precision_gb300 import build
    env = dict(os.environ, F8_LIBRARY=build.build(checked=True))
    tests = ["tests/test_gpu_gemm_act.py", "tests/test_gpu_rope.py", "tests/test_gpu_residual_norm.py",
             "tests/test_gpu_block_nn.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "-k", "not past_2_31", *tests], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=900)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m is not None and int(m.group(1)) >= 300, tail
