"""The bench's one line: every key that is read from it, and short enough to be read whole (no GPU)."""
import argparse
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("bench_under_test", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def record(bench, name, k):
    """A record of the size that a run on the GPU leaves: rooflines of every family, figures of every layer."""
    roof = {"bound": "alu", "achieved": 29.04 + k, "peak": 78.3, "unit": "TFLOP/s", "frac": 0.3708, "peak_source": "m" * 130,
            "work": "valid-tap FMAs x 2", "traffic": None, "kernel": "bwd_weight:large:f32", "calls": 12, "launches": 24,
            "ms": 22.0145, "share": 0.286}
    return {"workload": bench.WORKLOAD_TEXT[name], "name": name, "value": 51.147 + k, "unit": "TFLOP/s", "ms_per_step": 76.9676,
            "GBps": 427.3, "TFLOPs_valid": 51.147, "dtype": "f32+f16", "step_bytes": 32890109184, "step_fma_valid": 1968316416000,
            "roofline": roof, "roofline_by_family": {f"family{i}": roof for i in range(12)},
            "per_layer": {f"lk_H64_k{i}_f32": {"fwd": {"plan": "large", "us": 1.0, "GBps": 1.0, "TFLOPs": 1.0}} for i in range(60)},
            "gpu_launches": 60 + k, "clock_lines": [], "wall_s_timed": 1.0, "steps": 3,
            "e2e": {"value": 44.167 + k, "unit": "TFLOP/s", "ms_per_step": 89.1, "h2d_bytes_per_step": 10963369728,
                    "d2h_bytes_per_step": 10963369728, "copies": "c" * 90},
            "graph_replay": {"value": 51.4, "ms_per_step": 76.5}, "cpu_baseline": {"value": 0.027, "sample": "s" * 90}}


def test_the_line_is_whole(bench):
    args = argparse.Namespace(steps=20, warmup=5, layers="", batch=0)
    recs = {n: record(bench, n, k) for k, n in enumerate(bench.ORDER)}
    assert len(json.dumps(recs)) > 30_000
    text = json.dumps(bench.metric_line(args, recs, bench.HEADLINE, 1, 78.3))
    assert len(text) < 8_000 and "\n" not in text
    line, head = json.loads(text), recs[bench.HEADLINE]
    for key in ("value", "unit", "ms_per_step", "dtype", "roofline", "e2e", "gpu_launches", "cpu_baseline"):
        assert line[key] == head[key]
    assert line["metric"] == bench.METRIC and line["config"]["name"] == bench.HEADLINE
    assert (line["n_gpus"], line["steps"], line["warmup"], line["higher_is_better"], line["scaling"]) == (1, 20, 5, True, "weak")
    assert line["gpu_launches_all_workloads"] == sum(r["gpu_launches"] for r in recs.values())
    assert {"vs_baseline", "data", "clocks"} <= set(line)
    for n, r in recs.items():
        s = line["configs"][n]
        assert (s["value"], s["ms_per_step"], s["e2e"], s["roofline"]["frac"]) == (r["value"], r["ms_per_step"], r["e2e"]["value"], 0.3708)


def test_records_of_a_shorter_run(bench):
    """Without the end-to-end pass, the graph or the CPU baseline those figures are null, or absent."""
    args = argparse.Namespace(steps=3, warmup=3, layers="a", batch=2)
    r = record(bench, "pr1", 0)
    r["e2e"] = r["graph_replay"] = None
    del r["cpu_baseline"]
    line = bench.metric_line(args, {"pr1": r}, "pr1", 2, 78.3)
    assert line["e2e"] is None and "cpu_baseline" not in line and line["n_gpus"] == 2
    assert line["configs"]["pr1"]["e2e"] is None and line["config"]["layers"] == "a" and line["config"]["batch_override"] == 2
