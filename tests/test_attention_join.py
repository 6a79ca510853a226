"""The join of attention over a cache of codes follows what the kernel before it left in memory, which a kernel that gave
up a wait may not have filled: join_check.cpp shows, on the host, that what it accepts stays within its buffers."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_heads_lead_nowhere_but_into_the_buffers(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "join_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-o", exe, os.path.join(HERE, "join_check.cpp")], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout
