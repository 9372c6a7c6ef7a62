"""The host half of the linear layer, the join and dropout under AddressSanitizer and UndefinedBehaviorSanitizer, as
test_host_sanitize.py does it for the block: tests/host_check_sublayer.cpp with the library's host sources, on the CPU."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from test_host_sanitize import CSRC, HOST_SOURCES, ROOT, _rocm

CSRC_OPS = os.path.join(ROOT, "activation_sparse_ffn_03_amd", "csrc_ops")


def test_sublayer_host_half_under_sanitizers(tmp_path):
    gxx, rocm = shutil.which("g++"), _rocm()
    if gxx is None or rocm is None:
        pytest.skip("needs g++ and the ROCm headers / runtime library")
    exe = str(tmp_path / "host_check_sublayer")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", CSRC_OPS,
           "-I", os.path.join(ROOT, "tests"), "-x", "c++"]
    cmd += [os.path.join(CSRC, s) for s in HOST_SOURCES] + [os.path.join(CSRC_OPS, s) for s in ("linear_api.hip", "join_api.hip")]
    cmd += [os.path.join(ROOT, "tests", "host_check_sublayer.cpp"), "-L", os.path.join(rocm, "lib"), "-lamdhip64",
            f"-Wl,-rpath,{os.path.join(rocm, 'lib')}", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"build failed:\n{r.stdout}\n{r.stderr}"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1",
               HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, f"host check failed (rc {r.returncode}):\n{r.stdout}\n{r.stderr[-6000:]}"
    assert "host check ok" in r.stdout
