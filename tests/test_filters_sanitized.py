"""The argument checks of the sampling, filtered-statistics and gradient-clipping
entry points (test_filters_cpu.py) against the library built with its host code
under AddressSanitizer and UndefinedBehaviorSanitizer.  Runs without a GPU."""
import os
import subprocess
import sys

import pytest

from test_abi_sanitized import ROOT, _runtime


def test_filter_checks_under_sanitizers():
    import torch

    if torch.cuda.is_available():
        pytest.skip("host-only check: the argument tests use made-up device pointers")
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not (asan and ubsan):
        pytest.skip("gcc sanitizer runtimes not found")
    from vocab_wide_token_gb300 import build

    try:
        lib = build.build_sanitized()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolchain for the sanitizer build: {e}")
    env = dict(os.environ, LD_PRELOAD=f"{asan}:{ubsan}", PSTAT_TEST_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-k", "argument",
                        os.path.join(ROOT, "tests", "test_filters_cpu.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out
