"""The host code of the 8-bit linear layers under AddressSanitizer and
UndefinedBehaviorSanitizer, with launchers that check every descriptor they
are given (tests/sanitize/q8_check.cpp): coverage of outputs and k, the
workspace's use, and that no buffer resource of the tile kernels passes its
operand. Built with g++ on the CPU, no device code."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "newton_schulz_04_amd", "csrc")
ROCM = "/opt/rocm"


def test_q8_host_code_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are missing")
    exe = str(tmp_path / "q8_check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                    f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "ns_q8_api.cpp"),
                    os.path.join(HERE, "sanitize", "q8_check.cpp"), "-o", exe, f"-L{ROCM}/lib",
                    f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64"], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "q8_check ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
