"""The windowed attention and the read-back on the bounds-checked build: their own tests run in
a child process with libisoq_checked.so, whose kernels compare every index with its extent;
each test there ends with the status word clear."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("name,pick", [
    ("test_gpu_window.py", "decode_window or chunk_window"),
    ("test_gpu_dequantize.py", "token_lists or rope_taken_off or long_lists or out_of_range")])
def test_checked_build_runs_clean(name, pick):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    lib = os.path.join(os.path.dirname(TESTS), "rotated_bit_kv_isoquant_b200", "libisoq_checked.so")
    if not os.path.exists(lib):
        pytest.skip("libisoq_checked.so not built")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(TESTS, name), "-x", "-q", "-m", "gpu",
                        "-k", pick], env=dict(os.environ, ISOQ_CHECK_BOUNDS="1"), capture_output=True,
                       text=True, timeout=600, cwd=os.path.dirname(TESTS))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
