"""Host-side checks of the training step's entry points under the address and
undefined-behaviour sanitizers (CPU only): refusals, workspace queries, and the
arguments that accepted calls hand to their kernels (tests/asan/train_asan.cpp)."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="needs g++ and hipcc")
def test_training_step_host_code_under_sanitizers(tmp_path):
    sys.path.insert(0, os.path.join(ROOT, "tests", "asan"))
    try:
        import build_train
    finally:
        sys.path.pop(0)
    exe = build_train.build(str(tmp_path / "build"))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    p = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env, timeout=600)
    assert p.returncode == 0, p.stdout[-4000:]
    assert "Sanitizer" not in p.stdout and "runtime error" not in p.stdout, p.stdout[-4000:]
    assert "all host checks passed" in p.stdout
