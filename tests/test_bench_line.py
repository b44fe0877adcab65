"""The line that bench.py prints: short enough to survive a reader that keeps only the end of a log, with every
field that a run is judged by."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
import inputgen  # noqa: E402

LIMIT = 4000
REASONS = ["hw_slowdown", "hw_thermal_slowdown", "sw_power_cap", "sw_thermal_slowdown"]
THIRD = 1e7 / 3  # a float with all of its digits


def _clocks():
    return {"sm_mhz": THIRD, "sm_min_mhz": 1372, "sm_max_mhz": 1965, "reasons": REASONS, "samples": 4000, "source": "NVML, 10 ms"}


def _record():
    """A record as long as any: every workload, all digits, all reasons, the longest texts."""
    wl = inputgen.WORKLOADS[bench.DEFAULT_WORKLOAD]
    stages = {s: THIRD for s in bench.STAGES}
    roof = {"kernel": "k" * 90, "bound": "tensor", "achieved": THIRD, "peak": THIRD, "unit": "TFLOP/s", "frac": THIRD,
            "algorithmic_flops_per_launch": 1.9e12, "kernel_ms": THIRD, "peak_source": "measured burst", "traffic": THIRD,
            "timing": "t" * 200}
    e2e = {"value": THIRD, "unit": "tokens/s", "h2d_bytes_per_step": 33554432, "d2h_bytes_per_step": 33554432,
           "us_per_call": THIRD, "pipelined_value": THIRD, "how": "h" * 200}
    entry = {"us_per_call": THIRD, "tokens_per_s": THIRD, "calls": 4000, "stat": "s" * 100, "us_p10": THIRD, "us_p90": THIRD,
             "roofline": roof, "stage_us_median": stages, "profiled_over_timed": THIRD, "e2e": e2e, "kernels_per_call": 7,
             "clocks": _clocks(), "clocks_profiled": _clocks(), "routing_counts": [1024] * 128, "config": bench.config_of(wl)}
    return {"metric": bench.METRIC, "value": THIRD, "unit": "tokens/s", "n_gpus": 8, "steps": 50, "warmup": 5,
            "ms_per_step": THIRD, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic (seeded SplitMix64 + Box-Muller inputs, random-init weights)",
            "config": dict(bench.config_of(wl), l2="inputs larger than L2: 2.82 GB of expert weights per step",
                           parallelism="replicas x8"),
            "roofline": roof, "e2e": e2e, "gpu_launches": 35000, "clocks": _clocks(), "clocks_profiled": _clocks(),
            "stage_ms_per_call": stages, "profiled_over_timed": THIRD, "stage_timing": "x" * 100,
            "median_ms_per_step": THIRD, "tflops_per_gpu_layer": THIRD, "routing_counts": [1024] * 128,
            "cpu_baseline": {"value": THIRD, "unit": "tokens/s", "cores": 1, "kind": "oracle", "sample": "s" * 250, "seconds": THIRD},
            "workloads": {name: entry for name in bench.ENTRY_WORKLOADS}}


def test_the_line_is_short():
    text = bench.printed(_record())
    assert len(text) <= LIMIT and "\n" not in text


def test_the_line_keeps_what_a_run_is_judged_by():
    rec = _record()
    line = json.loads(bench.printed(rec))
    for key in ("metric", "unit", "n_gpus", "steps", "warmup", "higher_is_better", "scaling", "vs_baseline", "dtype", "data",
                "config", "gpu_launches"):
        assert line[key] == rec[key], key
    for key in ("value", "ms_per_step"):
        assert abs(line[key] - rec[key]) <= 1e-7 * rec[key]
    assert set(line["e2e"]) >= {"value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"}
    assert set(line["clocks"]) == {"sm_mhz", "sm_max_mhz", "reasons"} and line["clocks"]["reasons"] == REASONS
    assert set(line["workloads"]) == set(bench.ENTRY_WORKLOADS)
    for entry in line["workloads"].values():
        assert set(entry) == {"us_per_call", "tokens_per_s", "roofline", "e2e", "clocks"}
        assert abs(entry["roofline"]["frac"] - THIRD) <= 1e-4 * THIRD


def test_rounding_reaches_every_float():
    assert bench.rounded({"a": [1.23456789, {"b": 2}], "c": "x", "d": None, "e": True}, 3) == {"a": [1.23, {"b": 2}], "c": "x",
                                                                                               "d": None, "e": True}
