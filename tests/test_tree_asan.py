"""The argument validation of drafted trees and of caches whose tokens carry their own scales under AddressSanitizer, on
the CPU: the ABI layers' host code, with stubs in place of the kernels' launchers (``tests/asan/tree_validation.cpp``)."""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_abi_asan import CSRC, FLAGS, HIPCC, ROOT, _run

DRIVER = os.path.join(ROOT, "tests", "asan", "tree_validation.cpp")
SOURCES = ("dspark_cache_abi.hip", "dspark_tree_abi.hip")


def test_validation_paths_under_address_sanitizer(tmp_path):
    if not os.path.exists(HIPCC) or shutil.which("nm") is None:
        pytest.skip("hipcc not available")
    objs = [str(tmp_path / (s[:-4] + ".o")) for s in SOURCES]
    cmds = [[HIPCC, *FLAGS, "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objs)]
    drv = str(tmp_path / "driver.o")
    cmds.append([HIPCC, *FLAGS, "-x", "hip", "-c", DRIVER, "-o", drv])
    with ThreadPoolExecutor(len(cmds)) as ex:
        list(ex.map(_run, cmds))
    exe = str(tmp_path / "tree_validation")
    _run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-o", exe, drv, *objs,
          "-L/opt/rocm/lib", "-lrocprofiler-sdk-roctx", "-Wl,-rpath,/opt/rocm/lib"])
    syms = subprocess.run(["nm", exe], capture_output=True, text=True, check=True).stdout
    assert "__asan_report_load" in syms  # the objects really are instrumented
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.stdout[-2000:], r.stderr[-2000:])
