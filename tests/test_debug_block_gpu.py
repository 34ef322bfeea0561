"""GPU: the tests of integer products and of gradients from 8-bit values through the checked
library (GEMM_DEBUG); each module ends by reading the device status, so a failed check fails it."""
import os
import subprocess
import sys

import pytest

from gpu_util import require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("module", ["test_linear_int8_gpu.py", "test_saved_backward_gpu.py", "test_eight_bit_block_gpu.py"])
def test_checked_library_runs_the_operators(module):
    require_gpu()
    subprocess.run([sys.executable, "-m", "dense_gemm_gb300.build", "--debug"], cwd=ROOT, check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.join("tests", module)],
                       cwd=ROOT, env=dict(os.environ, GEMM_LIBRARY="debug"), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "device check failed" not in r.stdout + r.stderr
