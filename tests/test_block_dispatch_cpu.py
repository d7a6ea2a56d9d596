"""The C ABI of the linear layer's and the router's calls past its refusals (api_linear.cpp, api_moe.cpp), built with
g++ under AddressSanitizer and UndefinedBehaviorSanitizer against a stand-in device and recording launchers (no GPU)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CSRC = "w4a16_int4_weight_linear_amd/csrc"


def test_dispatch_workspaces_and_shared_memory(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("g++ is required for the sanitizer build")
    exe = tmp_path / "block_dispatch_driver"
    srcs = [os.path.join(ROOT, p) for p in ("tests/sanitize/block_dispatch_driver.cpp",
                                            "tests/sanitize/block_recording_launchers.cpp", f"{CSRC}/api_linear.cpp",
                                            f"{CSRC}/api_moe.cpp")]
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", *srcs, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "block dispatch driver: ok" in r.stdout
