"""Routing's larger LDS is asked for on the device that a call runs on (no GPU: the HIP calls of
the library are taken by a library of this test, which writes them down)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r"""
#include <stddef.h>
#include <stdio.h>
typedef struct { unsigned x, y, z; } dim3_;
static dim3_ g, b; static size_t sh; static void* st;
int hipFuncSetAttribute(const void* f, int attr, int value) { printf("attribute %p %d\n", f, value); fflush(stdout); return 0; }
int __hipPushCallConfiguration(dim3_ grid, dim3_ block, size_t shared, void* stream) { g = grid; b = block; sh = shared; st = stream; return 0; }
int __hipPopCallConfiguration(dim3_* grid, dim3_* block, size_t* shared, void** stream) { *grid = g; *block = b; *shared = sh; *stream = st; return 0; }
int hipLaunchKernel(const void* f, dim3_ grid, dim3_ block, void** args, size_t shared, void* stream) { printf("launch %p %zu\n", f, shared); fflush(stdout); return 0; }
int hipGetLastError(void) { return 0; }
"""

CALLS = """
from bit_quantized_gemm_w4a16_amd import hq
for experts, groups in ((4095, 63), (4095, 63), (256, 8), (1030, 5), (4096, 64)):
    d = hq.route_desc(hq.HQ_DT_FP32, experts, 4, groups=groups, top_groups=2)
    hq.hq_moe_route(d, 3, 1 << 20, experts, None, 2 << 20, 3 << 20, stream=0)
"""


def test_each_call_that_needs_it_asks_for_the_lds(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "stub.c").write_text(STUB)
    subprocess.run([cc, "-shared", "-fPIC", "-O1", str(tmp_path / "stub.c"), "-o", str(tmp_path / "stub.so")], check=True)
    env = dict(os.environ, LD_PRELOAD=" ".join(filter(None, [str(tmp_path / "stub.so"), os.environ.get("LD_PRELOAD", "")])))
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-3000:]
    lines = [l.split() for l in r.stdout.splitlines() if l.split()[:1] in (["attribute"], ["launch"])]
    assert sum(l[0] == "launch" for l in lines) == 5, lines
    for i, l in enumerate(lines):
        # (3136 bytes are the kernel's own; 64 KB need no asking)
        if l[0] == "launch" and int(l[2]) + 3136 > 65536:
            before = lines[i - 1]
            assert before[0] == "attribute" and before[1] == l[1] and int(before[2]) >= int(l[2]), lines
    assert sum(int(l[2]) > 60000 for l in lines if l[0] == "launch") == 2
