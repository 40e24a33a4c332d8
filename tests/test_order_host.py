"""Tests that rely on a process's first queue run before those that use a second one, whatever the order of files (CPU only)."""

import os
import subprocess
import sys

from conftest import FIRST_QUEUE, ROOT


def test_first_queue_tests_come_first():
    files = ["tests/test_gpu_streams.py", "tests/test_gpu_newton_schulz.py", "tests/test_gpu_gemm.py"]
    out = subprocess.run([sys.executable, "-m", "pytest", "--collect-only", "-q", *files], cwd=ROOT, check=True,
                         stdout=subprocess.PIPE, text=True, env={**os.environ, "PYTHONDONTWRITEBYTECODE": "1"}).stdout
    names = [ln.split("::")[1].split("[")[0] for ln in out.splitlines() if "::" in ln]
    first = names.count(FIRST_QUEUE)
    assert first == 5 and names[:first] == [FIRST_QUEUE] * first
    assert {"test_fp8_and_newton_schulz_outputs", "test_sizes"} <= set(names[first:])
