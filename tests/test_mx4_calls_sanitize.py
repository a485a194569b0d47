"""The host side of the 4-bit calls under UndefinedBehaviorSanitizer:
tests/sanitize/mx4_calls_sanitize.cpp is built with the two HIP sources' host
pass (no device code) and calls them with arguments from the ends of every
range; HIP itself is replaced by stubs."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fsdp_sharded_state_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def test_checks_of_the_4bit_calls_clean_under_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("no HIP compiler")
    san = ["-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined"]
    objects = []
    for src in (os.path.join(CSRC, "fs_mx4.hip"), os.path.join(CSRC, "fs_mx4_matmul.hip"), os.path.join(CSRC, "fs_plan.cpp"),
                os.path.join(ROOT, "tests", "sanitize", "mx4_calls_sanitize.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, "-x", "hip", "-std=c++17", "-O1", "-g", "--offload-arch=gfx950", "--offload-host-only", *san, "-c", src, "-o", obj],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        objects.append(obj)
    exe = str(tmp_path / "mx4_calls_sanitize")
    # (there is no device code, whose place the host objects name)
    r = subprocess.run([os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "llvm", "bin", "clang++"), "-fsanitize=undefined",
                        *objects, "-Wl,--unresolved-symbols=ignore-all", "-no-pie", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=4"))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr, r.stderr[-4000:]
    assert r.stdout.strip().startswith("ok:"), r.stdout
