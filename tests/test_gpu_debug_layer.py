"""The batched layer through the bounds-checked build (libtcq_debug.so).

The tests of the products, gradients and 8-bit checkpoints (ragged shapes, odd strides,
cut reductions, unaligned outputs and residuals) run once more in a process of its own with
TCQ_LIBRARY=debug, where every plain load and store of their kernels is checked against
its array and tests/conftest.py requires the device error word to stay clear after each
test."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("file", ["test_gpu_gemm.py", "test_gpu_gemm_ranges.py", "test_gpu_q8.py", "test_gpu_layer.py"])
def test_batched_layer_through_the_bounds_checked_build(file, cuda_device):
    from trellis_coded_weight_tcq_b200 import build

    build.build(debug=True)
    env = dict(os.environ, TCQ_LIBRARY="debug")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join("tests", file), "-m", "gpu", "-x", "-q",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=420)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " passed" in r.stdout
