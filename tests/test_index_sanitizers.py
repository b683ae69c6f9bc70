"""The host code of the index-driven re-layouts under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU; g++, host code only)."""
import os
import subprocess

from tests.test_sanitizers import CSRC, ROOT, SAN, run


def test_index_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "index_sanitize")
    subprocess.run(["g++", "-std=c++17", "-DBASP_HD="] + SAN +
                   ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
                   + [os.path.join(CSRC, f) for f in ("plan.cpp", "launch.cpp", "index_plan.cpp")]
                   + [os.path.join(ROOT, "tests", "sanitize", "index_sanitize.cpp"), "-o", exe], check=True)
    run(exe)
