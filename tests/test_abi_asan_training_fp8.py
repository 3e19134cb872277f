"""The host code of the router's training pass and of the block-scaled 8-bit
operators under AddressSanitizer and with traps on undefined behaviour (CPU
only): `abi_host_training_fp8.cpp` drives sizes up to the largest ints through
workspaces, plans and calls that end at the last argument check.  The device
code is compiled as usual, without either."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                                reason="needs ROCm's hipcc and clang++")


def test_sizes_up_to_the_largest(tmp_path):
    lib, exe = tmp_path / "libtraining_fp8.so", tmp_path / "abi_host_training_fp8"
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "moe_gate_up_amd", "csrc")]
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fsanitize-trap=undefined", "-Xarch_host", "-fno-omit-frame-pointer", *inc,
                    *[os.path.join(ROOT, "moe_gate_up_amd", "csrc", src) for src in ("balance.hip", "block_fp8.hip")],
                    "-o", str(lib)], check=True, capture_output=True, timeout=600)
    subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fno-omit-frame-pointer",
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "abi_host_training_fp8.cpp"),
                    str(lib), f"-Wl,-rpath,{tmp_path}", "-o", str(exe)],
                   check=True, capture_output=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=99")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.returncode, r.stdout[-4000:] + r.stderr[-4000:])
    assert ", 0 failures" in r.stdout
