"""The operators around the layer go on after a cudaDeviceReset (in a child process, whose own context it ends):
their kernels keep their shared-memory limits."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_calls_after_a_device_reset():
    r = subprocess.run([sys.executable, os.path.join(HERE, "device_reset_serve_process.py")], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "RESET_OK" in r.stdout, r.stdout + r.stderr
