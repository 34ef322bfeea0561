"""GPU: the kernels along rows (layer norm, its gradients, rows in 8 bits) through the checked
library: granules shared by neighbouring rows, copies whose addresses are stepped from row to row, the
ring used again for the column sums, and the partial sums' places. They are in a translation unit of
their own; the self-test shows that its failed checks are reported too."""
import os
import subprocess
import sys

import pytest

from gpu_util import require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked():
    require_gpu()
    subprocess.run([sys.executable, "-m", "dense_gemm_gb300.build", "--debug"], cwd=ROOT, check=True)
    return dict(os.environ, GEMM_LIBRARY="debug")


@pytest.mark.parametrize("module", ["test_layer_norm_gpu.py", "test_quantize_rows_gpu.py", "test_quantize_ties_gpu.py", "test_layer_norm_equal_rows_gpu.py",
                                    "test_layer_norm_backward_isolation_gpu.py", "test_empty_width_gpu.py"])
def test_checked_library_runs_the_rows(checked, module):
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.join("tests", module)],
                       cwd=ROOT, env=checked, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "device check failed" not in r.stdout + r.stderr


def test_a_failed_check_of_the_rows_is_reported(checked):
    child = "from dense_gemm_gb300 import selftest_check, sync_status; print(selftest_check(), sync_status(), sync_status())"
    r = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=checked, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.split() == ["0", "5", "0"], (r.stdout + r.stderr)[-3000:]
    assert r.stderr.count("device check failed at source line") == 2 and "of ops_rows.cu" in r.stderr
