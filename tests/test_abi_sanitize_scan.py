"""The host code of the C-ABI layer of the recurrence, the convolution and the cache
of parked states under AddressSanitizer and UndefinedBehaviorSanitizer (host side
only), with launchers that only count (tests/abi_sanitize_scan_stubs.cpp) and a C
driver of calls to be refused and calls at the largest sizes
(tests/abi_sanitize_scan_driver.c). CPU only."""

import os
import shutil
import subprocess

import pytest

from test_abi_sanitize import CLANG, CLANGXX, CSRC, HERE, INCLUDE, ROCM, SAN_HOST, _run


@pytest.mark.timeout(600)
def test_scan_abi_under_asan_and_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or os.path.join(ROCM, "bin", "hipcc")
    if not (os.path.exists(hipcc) and os.path.exists(CLANGXX)):
        pytest.skip("ROCm toolchain not found")
    out = lambda name: str(tmp_path / name)  # noqa: E731
    objects = [out("scan_api.o")]
    _run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", CSRC, "-Xclang",
          "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN_HOST, "-c", os.path.join(CSRC, "scan_api.hip"), "-o",
          objects[-1]])
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    objects.append(out("stubs.o"))
    _run([CLANGXX, "-x", "hip", "--cuda-host-only", "-D__HIP_PLATFORM_AMD__", "-O1", "-g", "-std=c++17", "-fPIC", "-I",
          INCLUDE, "-I", CSRC, *san, "-c", os.path.join(HERE, "abi_sanitize_scan_stubs.cpp"), "-o", objects[-1]])
    objects.append(out("driver.o"))
    _run([CLANG, "-O1", "-g", "-Wall", "-Werror", "-I", INCLUDE, "-D__HIP_PLATFORM_AMD__", "-I",
          os.path.join(ROCM, "include"), *san, "-c", os.path.join(HERE, "abi_sanitize_scan_driver.c"), "-o", objects[-1]])
    exe = out("driver")
    _run([CLANGXX, "-fsanitize=address,undefined", *objects, "-o", exe, "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
          "-Wl,-rpath," + os.path.join(ROCM, "lib")])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
