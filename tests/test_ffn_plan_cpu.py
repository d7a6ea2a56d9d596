"""The work splits of the feed-forward block's kernels (split_plan.hpp, gemm_t_skinny_plan.hpp),
swept on the host under AddressSanitizer and UndefinedBehaviorSanitizer: steps covered once,
parts where the join looks for them, 32-bit positions against 64 bits (no GPU)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def test_plans(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("g++ is required for the sanitizer build")
    exe = tmp_path / "plan_driver"
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", os.path.join(ROOT, "tests/sanitize/plan_driver.cpp"),
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "plan driver: ok" in r.stdout
