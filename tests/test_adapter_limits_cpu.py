"""The sizes that the adapters' kernels address with 32 bits (csrc/adapter_ops.hpp),
checked on the host by tests/sanitize/adapter_limits.hip.  No GPU is needed or touched.
"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
OUT = os.path.join(ROOT, "_build", "adapter_limits")


def test_what_is_addressed_with_32_bits_fits_them():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    os.makedirs(OUT, exist_ok=True)
    exe = os.path.join(OUT, "adapter_limits")
    src = os.path.join(ROOT, "tests", "sanitize", "adapter_limits.hip")
    res = subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", src, "-o", exe],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and ", 0 failed" in res.stdout, res.stdout
