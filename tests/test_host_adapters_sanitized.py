"""The host code of the adapters' and dropout's entry points under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU, as test_host_sanitized does for the linears': each at
its smallest and largest shapes, formats and set sizes, on workspaces of exactly the size asked
for and shorter ones, with every recorded launch within the hardware's limits."""

import concurrent.futures as cf
import os
import shutil
import subprocess

import pytest

import test_host_sanitized as H

KERNELS = H.KERNEL_SOURCES + ["adapters", "adapters_gemm", "dropout"]


def test_adapters_host_code_under_sanitizers():
    if not (shutil.which("g++") and os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs g++ and hipcc")
    os.makedirs(H.OUT, exist_ok=True)
    sources = [os.path.join(H.CSRC, n) for n in ("api.cpp", "codebook.cpp", "adapters_api.cpp")]
    sources += [os.path.join(H.HERE, n) for n in ("sim_runtime.cpp", "adapters_check.cpp")]
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        kern = list(ex.map(H._host_side, KERNELS))
        san = list(ex.map(H._sanitized, sources))
    exe = os.path.join(H.OUT, "adapters_check")
    H._run(["g++", *H.SAN, "-o", exe, *san, *kern, H._fatbin_stubs(kern), "-lpthread"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:abort_on_error=0:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-8000:]
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-8000:]
    last = r.stdout.splitlines()[-1]
    assert last.startswith("OK ") and int(last.split()[1]) > 10000, last
