"""The rows' division by their group of heads, on the CPU under the sanitizers."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_division_under_sanitizers(tmp_path):
    exe = str(tmp_path / "q8_divide_checks")
    r = subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fsanitize=undefined",
                        "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "sanitize", "q8_divide_checks.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and " 0 failure(s)" in r.stdout, (r.stdout + r.stderr)[-3000:]
