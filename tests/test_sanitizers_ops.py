"""The host side of the prompt, single-token and log-probability entry points, built with
AddressSanitizer and UndefinedBehaviorSanitizer, runs clean: every entry point accepted and
refused with the kernel launchers replaced by recording stubs, two threads refusing at once.
Built with g++ for the host only."""
import os
import shutil
import subprocess

import pytest

from tests.test_sanitizers import HERE, ROCM_INCLUDE, ROOT, SAN, _run


def test_ops_abi_validation_under_asan_and_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")):
        pytest.skip("no g++ or no HIP headers")
    exe = tmp_path / "ops_abi_driver"
    csrc = os.path.join(ROOT, "gated_delta_rule_rows_amd", "csrc")
    subprocess.run([cxx, "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "kda_ops_abi.cpp"), os.path.join(HERE, "ops_abi_driver.cpp"),
                    "-o", str(exe), "-pthread"], check=True)
    _run(exe)
