"""The rule for clusters of the single tokens' kernel, on the host.  Compiles tests/step_rule_check.cu with nvcc against
the in-tree library; no GPU needed."""
import os
import shutil
import subprocess

import pytest

from paged_kv_gqa_11_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_more_clusters_than_the_device_holds(tmp_path):
    nvcc = shutil.which("nvcc")
    if nvcc is None:
        pytest.skip("nvcc not on PATH")
    lib = _build.build()
    exe = str(tmp_path / "step_rule_check")
    cmd = [nvcc, *_build.ARCH, "-std=c++17", "-O2", "-I", _build.INCLUDE, "-I", _build.CSRC,
           os.path.join(HERE, "step_rule_check.cu"), "-o", exe, "-L", os.path.dirname(lib), "-lpa",
           "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)]
    done = subprocess.run(cmd, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and "mismatches 0" in out.stdout, out.stdout + out.stderr
