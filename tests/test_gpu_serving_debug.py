"""The suites of the operators around a serving step's attention, run again in
a child process against the bounds-checked debug library: they pass and leave
no record, beside data that the tests make bad on purpose."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("suite", ["test_gpu_rope.py", "test_gpu_verify.py", "test_gpu_pages.py", "test_gpu_serving_step.py"])
def test_serving_suites_under_debug_build(suite):
    env = dict(os.environ, CPATTN_DEBUG="1")
    probe = "import context_long_sequence_gb300 as c; assert c.cp_debug_build()"
    r = subprocess.run([sys.executable, "-c", probe], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.join("tests", suite)]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
