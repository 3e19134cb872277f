"""The host code of the calls around the experts under AddressSanitizer and with
traps on undefined behaviour (CPU only): `abi_host_around_experts.cpp` drives sizes up
to the largest ints through workspaces and calls that end at the last argument check.
The device code is compiled as usual, without either."""
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
    lib, exe = tmp_path / "libaround_experts.so", tmp_path / "abi_host_around_experts"
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "moe_gate_up_amd", "csrc")]
    objs = [str(tmp_path / f"{name}.o") for name in ("route_experts", "rms_norm", "rms_norm_backward", "adapters")]
    procs = [subprocess.Popen([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-c",
                               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                               "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                               "-Xarch_host", "-fsanitize-trap=undefined", "-Xarch_host", "-fno-omit-frame-pointer", *inc,
                               os.path.join(ROOT, "moe_gate_up_amd", "csrc", os.path.basename(o)[:-2] + ".hip"), "-o", o],
                              stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL) for o in objs]
    assert [p.wait(timeout=600) for p in procs] == [0] * len(procs)
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-Xarch_host", "-fsanitize=address", *objs, "-o", str(lib)],
                   check=True, capture_output=True, timeout=600)
    subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fno-omit-frame-pointer",
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "abi_host_around_experts.cpp"),
                    str(lib), f"-Wl,-rpath,{tmp_path}", "-o", str(exe)],
                   check=True, capture_output=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=99")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.returncode, r.stdout[-4000:] + r.stderr[-4000:])
    assert ", 0 failures" in r.stdout
