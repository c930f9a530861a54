"""The host code of layer norm, embedding, gradient norm and clipping (argument
validation, workspace sizing, the overlap check) under AddressSanitizer and
UndefinedBehaviorSanitizer: the validation suite passes without a report."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

import quantized_lora_merge_b200.build as qbuild

from .test_abi_sanitized import ROOT, _asan_runtime, _sanitized_library


def test_train_ops_host_code_under_sanitizers():
    asan = _asan_runtime()
    if asan is None or not Path(qbuild.NVCC).exists():
        pytest.skip("nvcc or gcc's sanitizer runtime is not installed")
    lib = _sanitized_library()
    env = dict(os.environ, LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0:alloc_dealloc_mismatch=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([sys.executable, str(ROOT / "tests" / "train_ops_sanitize_run.py"), str(lib)], env=env,
                         capture_output=True, text=True, timeout=900, cwd=str(ROOT))
    assert res.returncode == 0, (res.stdout[-2000:], res.stderr[-3000:])
    assert "passed" in res.stdout
    assert "runtime error" not in res.stderr and "AddressSanitizer" not in res.stderr
