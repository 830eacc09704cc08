"""The source's side's host code (checks, workspace sizes, launches) under
AddressSanitizer and UndefinedBehaviorSanitizer, as tests/test_sanitizers.py
does for the exchange's."""
import os
import subprocess
import sys

import pytest

from tests.test_sanitizers import ROOT, SAN, _runtime


def test_source_host_code_under_sanitizers(tmp_path):
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not asan or not ubsan:
        pytest.skip("gcc sanitizer runtimes not installed")
    lib, csrc = str(tmp_path / "libafd_hostfake_san.so"), os.path.join(ROOT, "combine_layout_amd", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-fPIC", "-shared", "-Wall", *SAN, f"-I{os.path.join(ROOT, 'include')}",
                           os.path.join(csrc, "afd_core.cpp"), os.path.join(csrc, "afd_backend_fake.cpp"), "-o", lib])
    env = dict(os.environ, LD_PRELOAD=f"{asan}:{ubsan}", AFD_HOSTFAKE_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:detect_odr_violation=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    proc = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                           "tests/test_source_host.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = proc.stdout[-3000:] + proc.stderr[-3000:]
    assert proc.returncode == 0, tail
    assert " passed" in proc.stdout, tail
