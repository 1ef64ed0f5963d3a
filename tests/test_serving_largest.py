"""The host side of the serving calls at the largest sizes they accept, under sanitizers and without a device."""

import os
import shutil
import subprocess

import pytest

from weight_decompression_amd import build_lib

HERE = os.path.dirname(os.path.abspath(__file__))


def test_largest_sizes_are_clean_under_sanitizers(tmp_path):
    try:
        hipcc = build_lib.hipcc_path()
    except RuntimeError:
        pytest.skip("needs hipcc")
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "serve_largest_host")
    san = [a for f in ("-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer")
           for a in ("-Xarch_host", f)]
    subprocess.run([hipcc, f"--offload-arch={build_lib.OFFLOAD_ARCH}", "-O1", "-g", "-std=c++17", "-Xarch_device", "-O1", *san,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", build_lib.INCLUDE, "-o", exe,
                    os.path.join(build_lib.CSRC_SERVE, "llvq_serve.hip"), os.path.join(HERE, "host_build", "serve_largest_host.cpp")],
                   check=True, capture_output=True)
    # no device is to be seen, wherever this runs
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1",
               HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert p.returncode == 0, p.stdout[-1000:] + p.stderr[-3000:]
    assert "runtime error" not in p.stderr and "AddressSanitizer" not in p.stderr, p.stderr[-3000:]
    assert p.stdout.startswith("ok ")
