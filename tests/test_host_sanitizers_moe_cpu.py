"""libgba_moe's host code under AddressSanitizer and UndefinedBehaviorSanitizer, as
tests/test_host_sanitizers_cpu.py has libgba's: gm_api.hip (argument checks, choice of kernel) compiled again
with both on its host side only, linked with the other objects of the current build and
tests/host_sanitize_moe.c, and run without a GPU."""
import glob
import os
import subprocess

import pytest

from tests.test_host_sanitizers_cpu import BUILD, CLANG, CLANGXX, CSRC, HIPCC, ROOT, SAN

MOE = os.path.join(CSRC, "moe")


def test_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    for tool in (HIPCC, CLANG, CLANGXX):
        if not os.path.exists(tool):
            pytest.skip("ROCm compilers not installed")
    objs = [os.path.join(BUILD, os.path.basename(s)[:-4] + ".o") for s in sorted(glob.glob(os.path.join(MOE, "*.hip")))
            if os.path.basename(s) != "gm_api.hip"]
    missing = [o for o in objs if not os.path.exists(o)]
    if missing:
        pytest.skip("library not built (run build() first): %s" % missing[0])
    api, prog, exe = (str(tmp_path / n) for n in ("gm_api_san.o", "check.o", "check"))
    include = "-I" + os.path.join(ROOT, "include")
    steps = [[HIPCC, "-O1", "-std=c++17", "-fPIC", "--offload-arch=gfx950", include, "-I" + CSRC,
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument"]
             + [f for flag in SAN for f in ("-Xarch_host", flag)] + ["-c", os.path.join(MOE, "gm_api.hip"), "-o", api],
             [CLANG, "-O1", include] + SAN + ["-c", os.path.join(ROOT, "tests", "host_sanitize_moe.c"), "-o", prog],
             [CLANGXX, "-fsanitize=address", "-fsanitize=undefined", prog, api] + objs
             + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-lm", "-o", exe]]
    for cmd in steps:
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
    syms = subprocess.run(["nm", api], capture_output=True, text=True, check=True).stdout
    assert "__asan_report" in syms and "__ubsan_handle" in syms      # really instrumented
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    if r.returncode == 77:
        pytest.skip(r.stdout.strip())
    report = r.stdout + r.stderr
    assert "AddressSanitizer" not in report and "LeakSanitizer" not in report, report[-6000:]
    assert "runtime error" not in report, report[-6000:]
    assert r.returncode == 0 and "host sanitize check ok" in r.stdout, report[-6000:]
