"""The speculative decode entry points under the address and
undefined-behaviour sanitizers, on the host: tests/native/speculative_sanitize.cpp
sizes workspaces over the ends of their ranges and makes calls that the host
checks must reject.  As in test_sanitize.py its fake device pointers never
reach a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

from test_sanitize import ROOT, _gpu_visible


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="needs hipcc")
@pytest.mark.skipif(_gpu_visible(), reason="host-only check: its fake device pointers must never reach a GPU")
def test_speculative_entry_points_under_sanitizers(tmp_path):
    sys.path.insert(0, os.path.join(ROOT, "tests", "native"))
    try:
        import build_sanitize as b
    finally:
        sys.path.pop(0)
    b.build(str(tmp_path))                      # the library's objects
    objs = sorted(str(o) for o in tmp_path.glob("*.o") if o.name != "abi_sanitize.o")
    clang, lib = os.path.join(b.ROCM, "llvm", "bin", "clang++"), os.path.join(b.ROCM, "lib")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    b._run([clang, "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I", b.INC, "-I", os.path.join(b.ROCM, "include"),
            *san, "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer",
            "-c", os.path.join(b.HERE, "speculative_sanitize.cpp"), "-o", drv])
    b._run([clang, *san, "-o", exe, drv, *objs, "-L", lib, "-lamdhip64", f"-Wl,-rpath,{lib}"])
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "all passed" in r.stdout
    assert "AddressSanitizer" not in out and "runtime error" not in out and "LeakSanitizer" not in out
