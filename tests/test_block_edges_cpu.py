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


def test_every_call_is_exported():
    """`from ... import *` brings each function of the binding that has no underscore."""
    import inspect

    import w4a16_int4_weight_linear_amd as w4
    calls = {n for n, f in inspect.getmembers(w4, inspect.isfunction) if not n.startswith("_") and f.__module__ == w4.__name__}
    assert calls - set(w4.__all__) == set()
    assert all(hasattr(w4, n) or hasattr(w4.lib, n) for n in w4.__all__)
