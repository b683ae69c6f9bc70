"""The 32-bit row arithmetic of the sort by expert at the largest sizes a plan
accepts, under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU; g++,
host code only)."""
import os
import subprocess

from tests.test_sanitizers import CSRC, ROOT, SAN, run


def test_rows_of_the_experts_at_the_limits(tmp_path):
    exe = str(tmp_path / "expert_rows_sanitize")
    subprocess.run(["g++", "-std=c++17", "-DBASP_HD="] + SAN +
                   ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
                   + [os.path.join(CSRC, f) for f in ("plan.cpp", "launch.cpp", "index_plan.cpp")]
                   + [os.path.join(ROOT, "tests", "sanitize", "expert_rows_sanitize.cpp"), "-o", exe], check=True)
    run(exe)
