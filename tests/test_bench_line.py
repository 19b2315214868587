"""The line that a default benchmark run prints (no GPU)."""
import json

import bench


def record(name, unit="TFLOP/s"):
    """A record as `report` makes them, every number with all the digits it may have."""
    row = {"M": 8192, "flops": 481036337152.0, "bytes": 199802880, "us": 123456.78, "us_p10": 123456.78, "us_p90": 123456.78, "tflops": 1199.14,
           "gbps": 12345.6, "hbm_frac": 0.123, "mfma_frac": 0.123, "roofline_frac": 0.123, "traffic_bytes": 8930055945, "traffic_ratio": 1.921}
    return {"metric": bench.METRIC, "value": 1020.66, "unit": unit, "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 0.9425,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "fp16", "data": "synthetic",
            "config": {"workload": name, "M_sweep": bench.SWEEP, "N": 4096, "K": 7168, "cold_weight_copies": 36},
            "roofline": {"bound": "mfma", "achieved": 1199.1, "peak": 2500.0, "unit": unit, "frac": 0.4797, "measured_peak": 2088.5,
                         "frac_of_measured": 0.5742, "traffic": 424599838, "kernel": "tile_gemm_kernel<WNA16_FP16> (M>64)", "M": 8192,
                         "avg_us": 401.15, "algorithmic_flops": 481036337152.0, "algorithmic_bytes": 199802880,
                         "per_unit": "2*M*N*K flops per launch"},
            "cpu_baseline": {"value": 0.001173, "unit": unit, "cores": 16, "kind": "oracle", "sample": "256 output rows x N=4096 x K=7168"},
            "per_M": [row] * len(bench.SWEEP)}


def test_the_line_is_short_enough_to_be_read_whole():
    """One line of a few KB that has the headline workload's record whole and every other workload's result."""
    head = record("dense_w4a16_zp_fp16_N4096_K7168")
    head["peaks"] = {k: {"measured": 6162.3, "unit": "GB/s", "spec": 8000.0, "frac_of_spec": 0.77} for k in ("hbm", "fp16", "bf16", "fp8", "fp4", "int8")}
    extra = {nm: record("moe_w4a16_mxfp4_indexed_E256_top8_N4096_K7168") for nm in bench.DEFAULT_EXTRA}
    line = bench.headline(head, extra)
    assert "\n" not in line and len(line) < 10000
    got = json.loads(line)
    assert {k: v for k, v in got.items() if k != "configs"} == head
    assert list(got["configs"]) == list(bench.DEFAULT_EXTRA)
    for rec in got["configs"].values():
        assert rec["value"] == 1020.66 and rec["ms_per_step"] == 0.9425 and rec["roofline_frac"] == 0.4797
