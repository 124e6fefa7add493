"""The host code of the attention half (include/mxq_attention.h) under AddressSanitizer and UndefinedBehaviorSanitizer: its host
tests run against a build of the library's host side with both, as test_host_sanitized.py does for mxq.h."""

import os
import subprocess
import sys

import pytest

from conftest import ROOT
from mx_bit_quantized_amd import _build


def test_attention_host_tests_pass_under_asan_and_ubsan(tmp_path):
    rt = _build.sanitizer_runtime()
    if not rt:
        pytest.skip("no clang AddressSanitizer runtime in this image")
    env = dict(os.environ, LD_PRELOAD=rt, MXQ_TEST_LIB=_build.build_host_sanitized(str(tmp_path / "libmxq_asan.so")),
               # leaks and allocator pairs of the interpreter are not the library's
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    files = [os.path.join(ROOT, "tests", n) for n in ("test_attn_abi_host.py", "test_attn_limits_host.py")]
    res = subprocess.run([sys.executable, "-m", "pytest", *files, "-q", "-p", "no:cacheprovider", "-k", "not refuses_cpu and not binding"],
                         cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert "AddressSanitizer" not in res.stdout and "runtime error:" not in res.stdout, res.stdout[-4000:]
    assert res.returncode == 0 and " passed" in res.stdout, res.stdout[-4000:]
