"""bench.py's result: one JSON line on stdout that a reader of the output's last 2.5 KB gets
whole, and the long reports beside it on stderr."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402
import workloads  # noqa: E402


def full_line():
    """A line of the size that a run makes: every number at full length."""
    x = 1.0 / 3
    rows = [dict(M=m, N=18432, K=7168, us=x, GBps=1e4 * x, frac_measured=x, cublas_us=x) for m in range(64)]
    return {"metric": bench.METRIC, "value": 6e3 + x, "unit": bench.UNIT, "n_gpus": 1, "steps": 4000, "warmup": 5,
            "ms_per_step": x, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic (seeded N(0,1) activations, N(0,1/K) weights)", "impl": "ours",
            "config": bench.workload_config(workloads.CHAIN, {
                "pdl": True, "graph": False, "fused_gemm_reduce": True, "l2_prefetch_blocks": 0,
                "l2_after_reduce_blocks": 16, "parallelism": "single"}),
            "hbm_frac_of_measured": x, "hbm_frac_of_nominal_8000": x,
            "roofline": {"text": "r" * 460}, "kernels": {"text": "k" * 150},
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "samples": 42, "reasons": ["sw_power_cap"]},
            "e2e": {"value": x, "unit": bench.UNIT, "h2d_bytes_per_step": 5275648, "d2h_bytes_per_step": 458752,
                    "ms_per_step": x, "steps": 500}, "gpu_launches": 36000,
            "cpu_baseline": {"value": x, "unit": bench.UNIT, "cores": 16, "kind": "oracle", "sample": "s" * 180,
                             "one_thread": {"value": x, "sample": "s" * 180}},
            "parity": {"text": "p" * 1300}, "configs": {"gemm": rows, "reduce": rows}}


def test_the_line_is_short_and_nothing_is_lost(capsys):
    line = full_line()
    before = json.loads(json.dumps(line))
    bench.print_result(line)
    out, err = capsys.readouterr()
    assert out.endswith("\n") and out.count("\n") == 1 and len(out) <= 2500
    head, report = json.loads(out), json.loads(err)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "e2e", "clocks", "gpu_launches", "roofline", "impl"):
        assert head[key] == before[key]
    assert report["parity"] == before["parity"] and report["configs"] == before["configs"]
    assert report["cpu_baseline_one_thread"] == before["cpu_baseline"]["one_thread"]
    assert head["cpu_baseline"]["value"] == before["cpu_baseline"]["value"]


def test_a_line_without_reports_prints_nothing_else(capsys):
    line = {k: v for k, v in full_line().items() if k not in ("parity", "configs", "cpu_baseline")}
    bench.print_result(line)
    out, err = capsys.readouterr()
    assert json.loads(out) == line and err == ""
