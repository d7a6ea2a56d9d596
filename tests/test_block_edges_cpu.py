"""The edges of the linear layer's, the router's and the few-token experts' calls, on the host (no GPU)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CSRC = "w4a16_int4_weight_linear_amd/csrc"


def test_sizes_at_the_edges(tmp_path):
    """Grids and spans of the largest sizes, under AddressSanitizer and UndefinedBehaviorSanitizer."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("g++ is required for the sanitizer build")
    exe = tmp_path / "block_edges_driver"
    srcs = [os.path.join(ROOT, p) for p in ("tests/sanitize/block_edges_driver.cpp",
                                            "tests/sanitize/block_recording_launchers.cpp", f"{CSRC}/api_moe.cpp",
                                            f"{CSRC}/api_linear.cpp")]
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", *srcs, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "block edges driver: ok" in r.stdout
