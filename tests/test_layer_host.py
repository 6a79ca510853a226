"""The compiled host side of the decoder-layer operators: which library it calls (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import fp8_block_scaled_fp8bs_gb300 as fp8bs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHECK = """
import sys
import fp8_block_scaled_fp8bs_gb300 as fp8bs
fp8bs.load(sys.argv[1])
fp8bs._load_host()
with open("/proc/self/maps") as f:
    print({line.split()[-1] for line in f if "libfp8bs" in line} == {sys.argv[1]})
"""


def test_host_side_calls_the_library_that_was_loaded(tmp_path):
    fp8bs.load()                                 # (built, if it was not)
    fp8bs._load_host()
    other = str(tmp_path / "libfp8bs_other.so")
    shutil.copy(fp8bs.LIB_PATH, other)
    out = subprocess.run([sys.executable, "-c", CHECK, other], cwd=ROOT, capture_output=True, text=True, check=True)
    assert out.stdout.strip() == "True"
