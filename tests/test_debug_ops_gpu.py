"""GPU: the operators' tests through the checked library (GEMM_DEBUG), whose
kernels check the bounds and alignment of their accesses, record a failed check
in the device status and skip the access. Each of the test modules ends by
reading that status, so a failed check fails it."""
import os
import subprocess
import sys

import pytest

from gpu_util import require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("module", ["test_linear_gpu.py", "test_linear_places_gpu.py", "test_linear_epilogue_gpu.py", "test_rms_norm_gpu.py", "test_norm_places_gpu.py", "test_mlp_block_gpu.py"])
def test_checked_library_runs_the_operators(module):
    require_gpu()
    subprocess.run([sys.executable, "-m", "dense_gemm_gb300.build", "--debug"], cwd=ROOT, check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", module)],
                       cwd=ROOT, env=dict(os.environ, GEMM_LIBRARY="debug"), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "device check failed" not in r.stdout + r.stderr
