"""The host code of the row operators under AddressSanitizer and UndefinedBehaviorSanitizer
(no GPU needed): their sources, with the sanitizers on the host side only, linked with the C
driver tests/host/rows_checks.c, which calls every entry point with sizes of every kind."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizers import CSRC, HIPCC, INCLUDE, ROOT, SAN, _run

SOURCES = ["permute.hip", "route_backward.hip", "block_norm.hip", "runtime.hip"]


@pytest.mark.timeout(900)
def test_row_operators_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-fno-gpu-rdc",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", INCLUDE, "-I", CSRC] + SAN

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        _run([HIPCC] + flags + ["-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    drv = str(tmp_path / "rows_checks.o")
    _run([HIPCC, "-x", "c", "-O1", "-g", "-I", INCLUDE, "-c", os.path.join(ROOT, "tests", "host", "rows_checks.c"),
          "-o", drv])
    exe = str(tmp_path / "rows_checks")
    _run([HIPCC, "--offload-arch=gfx950", "-fno-gpu-rdc"] + SAN + ["-o", exe, drv] + objs)
    env = dict(os.environ)
    # the HIP runtime's own allocations live until exit: leaks are not checked
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=0"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert ", 0 failures" in r.stdout
