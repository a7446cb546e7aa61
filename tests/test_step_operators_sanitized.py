"""The host side of the operators around a tree's target pass under AddressSanitizer and UndefinedBehaviorSanitizer.

Their translation units are compiled with both sanitizers on the host code (the
device code as PTX only: no kernel runs here) and linked with
``step_operators_sanitize_driver.c``, which calls every entry point on the paths a
host without a usable GPU reaches.
"""
from __future__ import annotations

import os
import subprocess

import pytest

from tests.test_abi_sanitized import CSRC, HERE, INCLUDE, SANITIZE, _cuda_home


def test_step_operators_are_clean_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    cuda = _cuda_home()
    if cuda is None or not os.path.exists(os.path.join(cuda, "lib64", "libcudart.so")):
        pytest.skip("no nvcc or no shared CUDA runtime")
    xc = [a for f in SANITIZE for a in ("-Xcompiler", f)]
    objs, procs = [], []
    for unit in ("penalties", "cache", "attend"):
        objs.append(str(tmp_path / (unit + ".o")))
        procs.append(subprocess.Popen(
            [os.path.join(cuda, "bin", "nvcc"), "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-g", "-std=c++17",
             *xc, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, unit + ".cu"), "-o", objs[-1]],
            stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
    for p in procs:
        out, err = p.communicate()
        assert p.returncode == 0, err
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "step_operators_sanitized")
    for cmd in (["gcc", "-std=c11", "-O1", "-g", *SANITIZE, "-Wall", "-Wextra", "-Werror", "-I", INCLUDE, "-c",
                 os.path.join(HERE, "step_operators_sanitize_driver.c"), "-o", drv],
                ["g++", *SANITIZE, drv, *objs, "-L", os.path.join(cuda, "lib64"), "-lcudart",
                 "-Wl,-rpath," + os.path.join(cuda, "lib64"), "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 and ("lasan" in r.stderr or "lubsan" in r.stderr):
            pytest.skip("no sanitizer runtime on this host")
        assert r.returncode == 0, r.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(
        os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))
    assert run.returncode == 0 and "0 failed checks" in run.stdout, run.stdout + run.stderr
    assert "runtime error" not in run.stderr, run.stderr
