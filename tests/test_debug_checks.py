"""The debug build's checks: every kernel source has them (on the CPU), and the
paged-cache suites, run again against the debug library, pass and leave no
record: part rows, slots, token rows and TMA coordinates stay in bounds on
every shape there, beside data that the tests make bad on purpose."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_long_sequence_gb300", "csrc")
# cp_attn.cu has microbenchmarks and self-tests alone; ptx.cuh and debug.cuh no kernels.
KERNELS = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and f not in ("cp_attn.cu", "ptx.cuh", "debug.cuh") and
           re.search(r"__global__|__device__", open(os.path.join(CSRC, f)).read())]


@pytest.mark.parametrize("name", KERNELS)
def test_kernel_sources_check_their_accesses(name):
    assert "CP_IN_BOUNDS(" in open(os.path.join(CSRC, name)).read()


@pytest.mark.gpu
@pytest.mark.parametrize("suite", ["test_gpu_paged.py", "test_gpu_paged_use.py", "test_gpu_paged_data.py"])
def test_paged_suites_under_debug_build(suite):
    env = dict(os.environ, CPATTN_DEBUG="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.join("tests", suite)]
    probe = "import context_long_sequence_gb300 as c; assert c.cp_debug_build()"
    r = subprocess.run([sys.executable, "-c", probe], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
