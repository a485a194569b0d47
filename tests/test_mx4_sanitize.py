"""The planner of quantised shards under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/sanitize/mx4_plan_sanitize.cpp is built with
g++ (host code only) with fs_plan.cpp and fs_mx4_plan.cpp, and checks the tables
that the kernels index by."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fsdp_sharded_state_amd", "csrc")


def test_planner_of_quantised_shards_clean_under_asan_ubsan(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    exe = str(tmp_path / "mx4_plan_sanitize")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g", "-O1"]
    r = subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *san,
                        os.path.join(ROOT, "tests", "sanitize", "mx4_plan_sanitize.cpp"), os.path.join(CSRC, "fs_plan.cpp"),
                        os.path.join(CSRC, "fs_mx4_plan.cpp"), "-o", exe], capture_output=True, text=True)
    if r.returncode != 0 and "hip_runtime_api.h" in r.stderr:
        pytest.skip("HIP headers not available for a host build")
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=3:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=4")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.stdout.strip().startswith("ok:"), r.stdout
