"""bench.py's line on standard output: short enough for a reader who keeps the last 2000 characters,
with nothing of the record lost."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def record():
    row = {"GiB_per_s": 6134.56, "GiB_per_s_fastest": 6234.5, "median_us": 1234.56, "min_us": 1234.56, "batched_us": 1234.56,
           "pct_of_hbm_peak": 82.34, "pct_of_store_ceiling": 93.45, "bytes_written": 1 << 31, "bytes_read": 0, "kernels": 1}
    fills = [k for k in bench.FILL_KERNELS if not k.startswith("constant")] + [f"below_number_{k}" for k in range(9)]
    return {
        "metric": "GiB/s written per fill (2^28 elems) on 1 MI355X; % of HBM write peak", "value": 6134.56, "unit": "GiB/s",
        "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 3.6789, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "per fill: u8/u16/u32/u64 integers, f16/f32/f64", "data": "synthetic",
        "config": {"workload": "w" * 260, "elements_per_fill": 1 << 28, "fills_per_step": len(fills),
                   "bytes_written_per_step": 24159191040},
        "pct_of_hbm_peak": 82.34,
        "roofline": {"bound": "hbm", "kernel": "normal_f64", "achieved": 5982.6, "peak": 8000.0, "unit": "GB/s", "frac": 0.7478,
                     "traffic": 2224463239, "bytes_per_launch": 2147483648, "avg_launch_ms": 0.35895, "frac_of_store_ceiling": 0.8},
        "cpu_baseline": {"value": 0.6932604235121371, "unit": "GiB/s", "cores": 16, "kind": "oracle", "sample": "s" * 120,
                         "single_core": {"value": 0.1234, "cores": 1, "log2_elements": 24},
                         "per_fill": {k: {"all_cores_s": 1.23456, "single_core_s_scaled": 12.3456} for k in fills}},
        "protocol": {"a": "p" * 300}, "store_ceiling": {"rows": [row] * 12}, "fills": {k: dict(row) for k in fills},
        "per_start": {k: {"0": row, "1": row} for k in fills}, "store_pattern": {"x": row}, "next_rows": {"y": row},
        "device": {"name": "d"}}


def test_the_line_is_short_and_nothing_is_lost():
    rec = record()
    assert len(json.dumps(rec)) > 10000
    line, details = bench.split_record(rec)
    text = json.dumps(line)
    assert len(text) < 2000 and "\n" not in text
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
              "dtype", "data", "config", "roofline", "pct_of_hbm_peak"):
        assert line[k] == rec[k]
    assert line["fills_GiB_per_s"] == {k: v["GiB_per_s"] for k, v in rec["fills"].items()}
    for k, v in rec.items():
        if k == "cpu_baseline":
            assert {**line[k], "per_fill": details["cpu_baseline_per_fill"]} == v
        else:
            assert (details if k in bench.DETAILS else line)[k] == v


def test_a_run_without_the_baseline():
    line, details = bench.split_record({**record(), "cpu_baseline": None})
    assert line["cpu_baseline"] is None and "cpu_baseline_per_fill" not in details
