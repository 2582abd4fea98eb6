"""Offsets of buffer stores, without a GPU."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_06_amd", "csrc")


def test_rows_past_the_longest_sequences_stay_outside_the_buffer(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    exe = tmp_path / "offset_driver"
    src = os.path.join(ROOT, "tests", "sanitize", "offset_driver.cpp")
    out = subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", f"-I{CSRC}", src, "-o", str(exe)],
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-4000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout


def test_sixteen_byte_buffer_stores_have_no_scalar_offset():
    """The compiler does not wait between such a store and an instruction that overwrites its registers, so all go through
    one helper, which puts the whole offset into the lane's register."""
    found = {}
    for path in glob.glob(os.path.join(CSRC, "*")):
        if os.path.isfile(path):
            text = re.sub(r"//[^\n]*", "", open(path).read())
            calls = re.findall(r"raw_(?:ptr_)?buffer_store_b(?:96|128)\s*\(([^;]*)\);", text)
            if calls:
                found[os.path.basename(path)] = [re.sub(r"\s+", " ", c) for c in calls]
    assert found == {"chunk_layout.hpp": ["v, r, int(off), 0, 0"]}, found
