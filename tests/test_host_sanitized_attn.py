"""The host code of the attention half (include/mxq_attention.h) under AddressSanitizer and UndefinedBehaviorSanitizer: its host
tests run against the build that test_host_sanitized.py makes for those of mxq.h, in a child process with the sanitizer runtime
preloaded. Any report fails the test."""

import os
import subprocess
import sys

import pytest

from conftest import ROOT
from mx_bit_quantized_amd import _build

FILES = ("test_attn_abi_host.py", "test_attn_abi_range_host.py", "test_attn_limits_host.py")


def test_attention_host_tests_pass_under_asan_and_ubsan(tmp_path):
    rt = _build.sanitizer_runtime()
    if not rt:
        pytest.skip("no clang AddressSanitizer runtime in this image")
    env = dict(os.environ, LD_PRELOAD=rt, MXQ_TEST_LIB=_build.build_host_sanitized(str(tmp_path / "libmxq_asan.so")),
               # leaks and allocator pairs of the interpreter are not the library's
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    # (the binding's own checks never reach the library)
    res = subprocess.run([sys.executable, "-m", "pytest", *(os.path.join(ROOT, "tests", n) for n in FILES), "-q",
                          "-p", "no:cacheprovider", "-k", "not refuses_cpu and not binding"],
                         cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    out = res.stdout
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert res.returncode == 0, out[-4000:]
    assert " passed" in out, out[-2000:]
