"""The benchmark's line on stdout: whole, parsable, and short enough to survive where only the end of a log is kept."""
from __future__ import annotations

import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402


def _measured():
    """What a run measures, with legs as long as they get."""
    row = bench.direction_roofline(4 << 30, [1.1, 1.2, 1.3] * 10)
    legs = {"gather": dict(row), "scatter": dict(row)}
    link = dict(gbs=56.123456, link_gbs=57.123456, link_frac=0.981234, samples=[57.0] * 200)
    return {
        "metric": bench.METRIC, "value": 2940.12, "unit": "GB/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 2.9217,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "u8", "data": "synthetic",
        "config": {"workload": "w" * 300, "requests": 1, "max_request_tokens": 32768, "gpus": 1, "payload_bytes_each_way": 4 << 30,
                   "tiles_per_launch": 131072, "chunks": 128, "staging_bytes": 4 << 30},
        "roofline": {"bound": "hbm", "achieved": 5600.0, "peak": 8000.0, "unit": "GB/s", "frac": 0.7, "traffic": 8 << 30,
                     "kernel": "k" * 200, "directions": legs, "target_frac": 0.7, "below_target": [], "note": "n" * 1000},
        "cpu_baseline": {"value": 10.0, "sample": "s" * 300, "single_core": {"sample": "s" * 200}},
        "parity": {"gather": True, "scatter": True, "layers": "all 32"},
        "breakdown": legs, "d2d_memcpy_gbs": 4900.0, "small_calls": {"x": list(range(500))},
        "host_path": {"workload": "h" * 300, "gather": link, "scatter": link, "sweep_gbs": {str(i): link for i in range(20)},
                      "roofline": {"frac": 0.98}, "duplex": None},
        "other_workloads": {"workload_%d:token_major" % i: dict(legs, roofline={"frac": 0.7}) for i in range(16)},
        "layer_pipeline": {"x": [1.0] * 500}, "pool_placement": {"x": [1.0] * 500},
    }


def test_the_line_is_short_and_holds_the_contract():
    out = _measured()
    assert len(json.dumps(out)) > 10000
    line = bench.contract_line(out)
    assert "\n" not in line and len(line) < 6000
    got = json.loads(line)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
              "dtype", "data", "config", "cpu_baseline", "parity"):
        assert got[k] == out[k]
    assert got["roofline"]["frac"] == 0.7 and got["roofline"]["directions"] == out["roofline"]["directions"]
    assert got["host_path"] == {d: {"gbs": 56.1235, "link_gbs": 57.1235, "link_frac": 0.9812} for d in ("gather", "scatter")}
    assert len(got["other_workloads_hbm_frac"]) == 16


def test_the_line_of_a_run_without_its_other_legs():
    out = _measured()
    for k in ("cpu_baseline", "host_path", "other_workloads", "layer_pipeline", "pool_placement", "small_calls"):
        out[k] = None
    got = json.loads(bench.contract_line(out))
    assert got["value"] == 2940.12 and got["host_path"] == {} and got["other_workloads_hbm_frac"] == {}
