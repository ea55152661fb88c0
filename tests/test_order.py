"""The host-side tests of the C ABI pass in either order of their files."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("files", [("test_abi_products.py", "test_abi_host.py"), ("test_abi_host.py", "test_abi_products.py")])
def test_files_in_either_order(files):
    out = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                          *(os.path.join(HERE, f) for f in files)], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:]
