"""The host-side checks of the operators around BitLinear (csrc/block_api.hip)
and their work split (csrc/block_ops.hpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, built for the host only with every report fatal
(tests/sanitize/block_checks.hip stands in for the launchers).  No GPU is
needed or touched.
"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang++"
OUT = os.path.join(ROOT, "_build", "sanitize_block")
FLAGS = ["--offload-host-only", "-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer",
         "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=all",
         "-I", os.path.join(ROOT, "include")]


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, f"{' '.join(cmd)}\n{res.stdout}\n{res.stderr}"


def test_block_checks_clean_under_asan_and_ubsan():
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("the ROCm compilers are not installed")
    os.makedirs(OUT, exist_ok=True)
    objs = []
    for src in (os.path.join(ROOT, "bitlinear_absmean_ternarise_bit_amd", "csrc", "block_api.hip"),
                os.path.join(ROOT, "tests", "sanitize", "block_checks.hip")):
        objs.append(os.path.join(OUT, os.path.basename(src)[:-4] + ".o"))
        _run([HIPCC, *FLAGS, "-c", src, "-o", objs[-1]])
    exe = os.path.join(OUT, "block_checks")
    _run([CLANG, "-fsanitize=address,undefined", *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "Sanitizer" not in res.stderr, res.stderr
    assert ", 0 failed" in res.stdout and int(res.stdout.split()[0]) >= 1000
