"""libpa stands by itself: it builds, and the calls that go to it alone work,
where the Python module over it cannot be compiled (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import pytest

from paged_kv_gqa_11_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def tree(tmp_path):
    """A copy of the package whose objects are built already, except for the module."""
    _build.build()
    shutil.copytree(os.path.join(ROOT, "paged_kv_gqa_11_gb300"), tmp_path / "paged_kv_gqa_11_gb300")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    out = tmp_path / "paged_kv_gqa_11_gb300" / "_build"
    for f in os.listdir(out):
        if f.startswith("pa_calls"):
            os.remove(out / f)
    return tmp_path


def run(tree, code):
    return subprocess.run([sys.executable, "-c", code], cwd=tree, capture_output=True, text=True,
                          env={**os.environ, "PYTHONPATH": str(tree), "PYTHONDONTWRITEBYTECODE": "1"})


# nvcc and the linker replaced by ones that only leave their output, so that the test takes a second
FAKE = """
import subprocess, sys
real_popen, real_run = subprocess.Popen, subprocess.run
def out(cmd): return cmd[cmd.index('-o') + 1]
class Popen(real_popen):
    def __init__(self, cmd, **kw):
        if 'pa_calls.cpp' not in ' '.join(cmd): cmd = ['sh', '-c', 'echo > "$0"', out(cmd)]
        super().__init__(cmd, **kw)
subprocess.Popen = Popen
def run(cmd, **kw):
    if 'libpa.so' in out(cmd): open(out(cmd), 'w').write('linked'); return
    return real_run(cmd, **kw)
subprocess.run = run
from paged_kv_gqa_11_gb300 import _build
"""


def test_a_module_that_does_not_compile_leaves_the_library(tree):
    """Reported as an error, after the library is in its place; an older module, made for
    another library, is gone."""
    src = tree / "paged_kv_gqa_11_gb300" / "csrc" / "pa_calls.cpp"
    src.write_text("#error no such compiler\n")
    old = tree / "paged_kv_gqa_11_gb300" / "_build" / "pa_calls.so"
    old.write_text("old")
    os.remove(tree / "paged_kv_gqa_11_gb300" / "_build" / "libpa.so")
    r = run(tree, FAKE + "_build.build()")
    assert r.returncode != 0 and "pa_calls" in r.stderr, r.stderr
    assert not old.exists()
    assert (tree / "paged_kv_gqa_11_gb300" / "_build" / "libpa.so").read_text() == "linked"


def test_the_library_builds_without_torch(tree):
    os.remove(tree / "paged_kv_gqa_11_gb300" / "_build" / "libpa.so")
    r = run(tree, "import sys; sys.modules['torch'] = None\n" + FAKE + "_build.build()")
    assert r.returncode == 0, r.stderr
    assert (tree / "paged_kv_gqa_11_gb300" / "_build" / "libpa.so").read_text() == "linked"


def test_the_cache_needs_the_module_for_its_own_calls_only(tree):
    """Made without it; append_rope and the like say what is missing."""
    r = run(tree, """
import torch
zeros = torch.zeros
torch.zeros = lambda *a, device=None, **kw: zeros(*a, **kw)
from paged_kv_gqa_11_gb300.cache import PagedKVCache
from paged_kv_gqa_11_gb300.rope import Rope
c = PagedKVCache(4, 16, 8)
assert c.k_pool.numel() == 4 * 4 * 16 * 272
r = Rope([0.5] * 8)
for call in (lambda: c.read_rows(None, None, None), lambda: c.append_rope(r, None, None, None, None, None), lambda: r.apply(None, None, None),
             lambda: c.decode_prefix(None, None, None, None, None, None, 1)):
    try:
        call()
    except RuntimeError as e:
        assert 'pa_calls is not built' in str(e), e
    else:
        raise SystemExit('no error')
""")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("what", ["torch", "python"])
def test_a_module_of_another_torch_or_python_is_not_current(tree, what):
    code = "from paged_kv_gqa_11_gb300 import _build\n"
    change = {"torch": "import torch; torch.__version__ = '0.0'\n", "python": "import sysconfig; f = sysconfig.get_config_var\n"
              "sysconfig.get_config_var = lambda k: 'other' if k == 'SOABI' else f(k)\n"}[what]
    out = tree / "paged_kv_gqa_11_gb300" / "_build"
    for f in os.listdir(os.path.join(ROOT, "paged_kv_gqa_11_gb300", "_build")):
        if f.startswith("pa_calls"):
            shutil.copy2(os.path.join(ROOT, "paged_kv_gqa_11_gb300", "_build", f), out / f)
    for base, _, files in os.walk(tree):  # the copy's sources are older than what was built
        for f in files:
            if "_build/" not in os.path.join(base, f) or f == "_build.py":
                os.utime(os.path.join(base, f), (1, 1))
    assert run(tree, code + "assert _build.up_to_date()").returncode == 0
    assert run(tree, change + code + "assert not _build.up_to_date()").returncode == 0
