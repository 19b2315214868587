"""Counted HBM bytes in the benchmark's records (no GPU): they stand for the kernels
that they were taken on, whatever else the library holds."""
import os
import shutil
from types import SimpleNamespace

import pytest

import bench
from bit_quantized_gemm_w4a16_amd import hq


@pytest.fixture
def tree(tmp_path):
    for d in ("bit_quantized_gemm_w4a16_amd", "include"):
        shutil.copytree(os.path.join(bench.ROOT, d), tmp_path / d, ignore=shutil.ignore_patterns("*.so", "__pycache__"))
    return tmp_path


@pytest.mark.parametrize("file,counts", [("csrc/k_attn.hip", False), ("csrc/k_kv.hip", False), ("csrc/hq_kv.h", False), ("csrc/hq_api.cpp", False),
                                         ("csrc/tile_gemm.hpp", True), ("csrc/skinny.hpp", True), ("csrc/k_moe.hip", True), ("csrc/hq_device.hpp", True),
                                         ("build.py", True)])
def test_the_key_is_of_the_quantized_layers_kernels(tree, file, counts):
    before = bench.kernel_source_hash(tree)
    assert before == bench.kernel_source_hash()
    with open(tree / "bit_quantized_gemm_w4a16_amd" / file, "a") as f:
        f.write("\n")
    assert (bench.kernel_source_hash(tree) != before) == counts


def test_figures_are_of_the_planned_launch(tmp_path, monkeypatch):
    """A figure is given where its kernel is the plan's, and not where the plan has another."""
    desc = bench._DRY["c2"]()
    plan = hq.hq_gemm_plan(desc, 16)[0]
    os.makedirs(tmp_path / "profiles")
    rec = '{"layer": {"source_hash": "%s", "per_M": {"16": {"kernel": "%s", "kernel_bytes": 1, "call_bytes": 1}, ' \
          '"32": {"kernel": "another", "kernel_bytes": 1, "call_bytes": 1}}}}'
    (tmp_path / "profiles" / "traffic.json").write_text(rec % (bench.kernel_source_hash(), plan))
    key = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "kernel_source_hash", lambda: key)
    work = SimpleNamespace(name="layer", desc=desc)
    assert bench._traffic(work, 16)["call_bytes"] == 1
    assert bench._traffic(work, 32) is None and bench._traffic(work, 64) is None
    assert bench._traffic(SimpleNamespace(name="another", desc=desc), 16) is None
