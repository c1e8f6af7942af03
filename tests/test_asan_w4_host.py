"""The host code of the experts in 4 bits and of the router under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only), as tests/test_asan_expert_host.py does for the expert block: the
sources with both sanitizers on the host side only, linked with tests/c_abi/asan_w4_host.c, every
call of which returns before any HIP call."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_top_id_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang"
SOURCES = ["moonep_api.hip", "moonep_plan.hip", "moonep_move.hip", "moonep_norm.hip", "moonep_w4.hip", "moonep_router.hip"]


@pytest.mark.skipif(not (shutil.which(HIPCC) and shutil.which(CLANG)), reason="needs the ROCm toolchain")
def test_w4_and_router_host_paths_under_sanitizers(tmp_path):
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    procs, objs = [], []
    for src in SOURCES:
        objs.append(str(tmp_path / (src + ".o")))
        cmd = [HIPCC, "-O1", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-c",
               "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
               "-Xarch_host", "-fno-omit-frame-pointer", *inc, os.path.join(CSRC, src), "-o", objs[-1]]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    for src, p in procs:
        _, err = p.communicate(timeout=600)
        assert p.returncode == 0, f"{src}:\n{err[-3000:]}"
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    host_san = ["-fsanitize=address,undefined", "-fno-omit-frame-pointer"]
    for cmd in ([CLANG, "-O1", "-g", "-std=c11", *host_san, "-D__HIP_PLATFORM_AMD__", *inc, "-I", "/opt/rocm/include",
                 "-c", os.path.join(ROOT, "tests", "c_abi", "asan_w4_host.c"), "-o", drv],
                [CLANG + "++", *host_san, drv, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib",
                 "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "asan w4 host ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
