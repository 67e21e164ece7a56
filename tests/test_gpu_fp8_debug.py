"""The linear layers on the bounds-checked build (libqvae_debug.so): every load's ring
place and weight row, every accumulator's columns and every output row is
checked before the access; each of the selected tests asserts
qvae_get_error() == 0 after its calls, so that a recorded failure fails it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


@pytest.mark.gpu
def test_linear_layers_pass_on_the_bounds_checked_build():
    from video_vae_decode_b200 import build as cuda_build

    env = dict(os.environ, QVAE_LIBRARY=cuda_build.build(debug=True))
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                          "tests/test_gpu_fp8.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = res.stdout[-3000:] + res.stderr[-2000:]
    assert res.returncode == 0, tail
    assert " passed" in res.stdout and "failed" not in res.stdout, tail
