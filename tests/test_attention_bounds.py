"""The cutting of an attention call into sequences (csrc/wal_seq.h) on the host, under
UndefinedBehaviorSanitizer: whatever starts and lens hold, the rows and tokens that
the kernels go through are among those that there are, and no sum overflows."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_any_starts_and_lens_stay_inside(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path / "seq_bounds")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                        "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "sanitize", "seq_bounds.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=120)
    if r.returncode != 0 and "ubsan" in r.stderr and "cannot find" in r.stderr:
        pytest.skip("the sanitizer runtime is not installed")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
