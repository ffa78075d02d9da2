"""Where a GPU is present, no test passes made-up addresses to the library."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUN = """
import sys, torch, pytest
torch.cuda.is_available = lambda: True
sys.exit(pytest.main(["-q", "-rA", *sys.argv[1:]]))
"""


@pytest.mark.parametrize("name", ["test_abi.py", "test_paged_abi.py", "test_sampled_abi.py", "test_rope_abi.py"])
def test_argument_checks_are_skipped(name):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("tried where there is no GPU")
    r = subprocess.run([sys.executable, "-c", RUN, os.path.join("tests", name)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert " passed" not in r.stdout.splitlines()[-1] and " skipped" in r.stdout.splitlines()[-1], r.stdout
