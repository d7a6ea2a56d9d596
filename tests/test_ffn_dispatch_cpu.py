"""The feed-forward block's C ABI past its refusals (api_ffn.cpp): the launcher that each call
reaches, workspaces, and operands that share memory, built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer against a stand-in HIP runtime and recording launchers (no GPU)."""

import os
import shutil
import subprocess

import pytest

import w4a16_int4_weight_linear_amd as w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CSRC = "w4a16_int4_weight_linear_amd/csrc"


def test_dispatch_and_shared_memory(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("g++ is required for the sanitizer build")
    exe = tmp_path / "ffn_dispatch_driver"
    srcs = [os.path.join(ROOT, p) for p in ("tests/sanitize/ffn_dispatch_driver.cpp",
                                            "tests/sanitize/recording_launchers.cpp", "tests/sanitize/fake_hip.cpp",
                                            f"{CSRC}/api.cpp", f"{CSRC}/api_ffn.cpp")]
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", *srcs, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "ffn dispatch driver: ok" in r.stdout


def test_overlap_is_a_status_of_its_own():
    assert w4.ERR_OVERLAP == 9 and b"OVERLAP" in w4.lib.w4a16_status_str(w4.ERR_OVERLAP)


def test_a_workspace_is_device_memory():
    with pytest.raises(ValueError, match="HIP device"):
        w4.ffn_workspace("gemm_t", 1, 1024, 1024, 128, device="cpu")
