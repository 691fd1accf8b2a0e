"""The argument checks of expert selection, block quantisation, 8-bit products and
the shared expert under AddressSanitizer and UndefinedBehaviorSanitizer
(test_host_checks.py has the build's description)."""
import os
import subprocess
import sys

import pytest

from routed_expert_prefill_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_dense_abi_under_host_sanitizers():
    rt = B.sanitizer_runtime()
    if rt is None:
        pytest.skip("the clang AddressSanitizer runtime is not installed")
    env = dict(os.environ, MOE_PREFILL_LIB=B.build_host_sanitized(), LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_dense_cpu.py")],
                       cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True, timeout=600)
    assert p.returncode == 0, p.stdout[-4000:]
    assert "passed" in p.stdout and "AddressSanitizer" not in p.stdout and \
        "runtime error" not in p.stdout, p.stdout[-4000:]
