import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and runs the CUDA library")
    config.addinivalue_line("markers", "slow: full-size parity case (minutes of host time)")


@pytest.fixture(scope="session")
def golden_dir():
    return os.path.join(ROOT, "tests", "golden")


# Their calls pass made-up addresses and rely on being refused; should a check let one through, it must end at the
# missing device and not in a kernel.
MADE_UP_ADDRESSES = ("test_abi.py", "test_paged_abi.py", "test_sampled_abi.py", "test_rope_abi.py")


@pytest.fixture(autouse=True)
def no_made_up_addresses_on_a_gpu(request):
    if request.path.name in MADE_UP_ADDRESSES:
        import torch

        if torch.cuda.is_available():
            pytest.skip("argument checks on made-up addresses run where there is no GPU")
