"""Where the appends put a new row, for words that need not be a page table, on the CPU: what does not fit together
is refused, and a place that is given lies among the request's own pages."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_word_at_its_ends(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ unavailable")
    inc = [os.path.join(ROOT, "decode_attention_append_gb300", "csrc"), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    exe = str(tmp_path / "place_check")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", *(f"-I{i}" for i in inc), os.path.join(ROOT, "tests", "place_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    n, found = map(int, r.stdout.split())
    assert n == 8 * 15 ** 5 * 9 and found > 1000
