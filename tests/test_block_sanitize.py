"""The host code of the operators around the experts (argument checks and
workspace sizes) under AddressSanitizer and UndefinedBehaviorSanitizer.

Their sources are compiled with both sanitizers on the host side, linked with
the library's other objects, and driven by tests/c/block_sanitize.c through calls that
the host answers alone (no GPU needed).  Any out-of-bounds access, leak or
undefined arithmetic aborts the run.
"""

import glob
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from int4_quantized_moe_amd import build as hip_build

from .conftest import ROOT
from .test_library_sanitize import HIPCC, SAN

SOURCES = ("kt_linear", "kt_router", "kt_ckpt8")


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("gcc") is None, reason="needs hipcc and gcc")
def test_block_host_code_clean_under_sanitizers(tmp_path):
    rest = [os.path.join(hip_build.OBJDIR, os.path.basename(s) + ".o")
            for s in sorted(glob.glob(os.path.join(hip_build.CSRC, "*.hip")))
            if os.path.basename(s)[:-4] not in SOURCES]
    if not all(os.path.exists(o) for o in rest):
        hip_build.build()

    def compile_one(name):
        obj = tmp_path / f"{name}.o"
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer", *SAN, "-Xclang",
                        "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-c",
                        os.path.join(hip_build.CSRC, f"{name}.hip"), "-o", str(obj)], check=True, capture_output=True)
        return str(obj)

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    driver = tmp_path / "block_sanitize.o"
    subprocess.run(["gcc", "-std=c11", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), "-c",
                    os.path.join(ROOT, "tests", "c", "block_sanitize.c"), "-o", str(driver)], check=True)
    exe = tmp_path / "block_sanitize"
    subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN[:4], *objs, *rest, str(driver), "-o", str(exe)], check=True,
                   capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    print(run.stdout[-3000:], run.stderr[-3000:])
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-2000:]
    assert "runtime error" not in run.stderr and "AddressSanitizer" not in run.stderr
    assert "FAIL" not in run.stdout and ", 0 failed" in run.stdout
