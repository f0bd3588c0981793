"""The host layer of the mixture-of-experts entry points under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): moe_api.cpp and
qmm_api.cpp with their kernel launchers stubbed out, driven by
tests/sanitize/moe_driver.cpp."""
import os
import shutil
import subprocess

import pytest

from test_sanitize import ROOT, SAN, _have_sanitizers


def test_moe_host_layer_under_sanitizers(tmp_path):
    if not shutil.which("gcc") or not shutil.which("g++"):
        pytest.skip("gcc / g++ not available")
    tmp = str(tmp_path)
    if not _have_sanitizers(tmp):
        pytest.skip("the compiler has no address / undefined-behaviour sanitizer runtime")
    csrc, san = os.path.join(ROOT, "quantized_matmul_ggml_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    objs = []
    for src in (os.path.join(csrc, "qmm_api.cpp"), os.path.join(csrc, "moe_api.cpp"), os.path.join(san, "host_stubs.cpp"),
                os.path.join(san, "moe_driver.cpp")):
        obj = os.path.join(tmp, os.path.basename(src) + ".o")
        r = subprocess.run(["g++", *SAN, "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-c", src, "-o", obj],
                           capture_output=True, text=True)
        assert r.returncode == 0, f"compile {src}:\n{r.stderr[-3000:]}"
        objs.append(obj)
    exe = os.path.join(tmp, "sanitized")
    r = subprocess.run(["g++", *SAN, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, f"sanitized run failed ({r.returncode}):\n{r.stdout[-2000:]}\n{r.stderr[-4000:]}"
    assert "runtime error" not in r.stderr and "ERROR: AddressSanitizer" not in r.stderr, r.stderr[-4000:]
