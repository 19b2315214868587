"""The host side of a routed layer's operators under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): their checks in hq_api.cpp and the layout
of the experts' workspace in k_moe_f8.hip, built with the sanitizers on the host
side alone, run through the host suite in a child process with every report fatal."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

import pytest

from test_sanitizers import CSRC, HIPCC, OUT, ROOT, _asan_runtime, _host_flags, _run

HOST = ("hq_api.cpp", "hq_repack.cpp", "k_moe_f8.hip")
SUITES = ["tests/test_layer_host.py"]


def _build() -> str:
    from bit_quantized_gemm_w4a16_amd import build as B

    os.makedirs(OUT, exist_ok=True)
    objs = []
    sources = [*glob.glob(os.path.join(CSRC, "*")), os.path.join(ROOT, "include", "hq.h"), B.__file__, __file__]
    newest = max(os.path.getmtime(f) for f in sources)
    for src in HOST:
        obj = os.path.join(OUT, "layer_" + src + ".o")
        objs.append(obj)
        if os.path.exists(obj) and os.path.getmtime(obj) > newest:
            continue
        # (B.COMMON's -O3 stays for the kernels)
        _run([HIPCC, "-x", "hip", *B.COMMON, "-g", *_host_flags(), "-Xarch_host", "-O1", "-c", os.path.join(CSRC, src), "-o", obj])
    for k in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        if os.path.basename(k) not in HOST:
            obj = os.path.join(B.BUILD, os.path.basename(k) + ".o")
            objs.append(obj if os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(k) else B._compile(k))
    lib = os.path.join(OUT, "libhq_layer.so")
    _run([HIPCC, f"--offload-arch={B.ARCH}", "-shared", "-fPIC", *_host_flags(), "-shared-libasan", *objs, "-o", lib])
    return lib


@pytest.mark.timeout(900)
def test_layer_host_code_under_asan_ubsan():
    runtime = _asan_runtime()
    if runtime is None or not os.path.exists(HIPCC):
        pytest.skip("clang's sanitizer runtime or hipcc not available")
    env = dict(os.environ)
    env.update({"LD_PRELOAD": runtime, "HQ_LIB_PATH": _build(),
                "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:detect_odr_violation=0:alloc_dealloc_mismatch=0",
                "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"})
    r = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-m", "not gpu", "-q", "-x", "-s", "-p", "no:cacheprovider"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=800)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-6000:]
    assert r.returncode == 0, out[-6000:]
    assert " passed" in r.stdout, out[-3000:]
