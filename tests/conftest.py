import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) and the CUDA library")
    config.addinivalue_line("markers", "slow: full-size cases, minutes of CPU or GPU time")


@pytest.fixture(autouse=True)
def no_device_error(request):
    """A wait that ran out, or a bounds check that failed on the checked build, fails the linear layers' test it happened
    in, not a later one."""
    yield
    if request.module.__name__.rpartition(".")[2] == "test_gpu_fp8":
        import torch
        from video_vae_decode_b200 import qvae

        if torch.cuda.is_available():
            torch.cuda.synchronize()
            assert qvae.qvae_get_error() == 0
