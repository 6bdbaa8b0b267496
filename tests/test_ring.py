"""How a block whose waits gave up leaves its ring of shared-memory slots, on
the CPU: tests/csrc/ring_check.cc compiles csrc/f8_ring.h, whose functions the
kernels call, and runs them on a model of the slots' mbarriers.  The copies
under way are waited for, each by its own phase, before the block leaves; no
slot is filled while its copy is under way."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_copy_has_landed(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "ring_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-o", str(exe),
                    os.path.join(HERE, "csrc", "ring_check.cc")], check=True)
    r = subprocess.run([str(exe), "20000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert " 0 mismatches" in r.stdout
