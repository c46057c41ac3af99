"""The line that bench.py prints is short enough for readers that keep the last few thousand characters of a run's output, and the
run's every field is on the other stream."""
import json
import types

import bench
import workload as wl

TEXT = "a sentence that says how a number was taken, as long as the longest of them are: " * 4


def full_line():
    """A line of the default run with every leg, each text and list as long as in earnest or longer."""
    roof = {"bound": "host_link", "achieved": 123.456789012345, "peak": 211.25605268485543, "unit": "GB/s", "frac": 0.61234567890123,
            "hbm_frac": 0.0123456789012345, "hbm_frac_of_nominal": 0.0104567890123456, "traffic": 123456789.5, "traffic_source": TEXT,
            "kernel": "hs_resolve_kernel", "kernel_ms_per_launch": 0.01234567890123, "launches": 1560, "timing": TEXT,
            "algorithmic_bytes_per_launch": {"link": 29123136.0, "hbm": 31523654.0}, "peak_source": TEXT}
    e2e = {"value": 197851.2345678901, "unit": bench.UNIT, "ms_per_step": 3.1539136000013457, "h2d_bytes_per_step": 262144,
           "d2h_bytes_per_step": 262144, "clock": TEXT, "path": TEXT, "out_slots_match_device_path": True, "median_ms": 3.15391360000134}
    cpu = {"value": 3068.077573273378, "unit": bench.UNIT, "cores": 1, "kind": "oracle", "sample": TEXT}
    one = {"workload": TEXT, "mode": "prefetch", "value": 528513.2918336492, "unit": bench.UNIT, "steps": 20, "ms_per_step": 1.23456789,
           "step_ms": [1.234567] * 20, "roofline": roof, "e2e": e2e, "host_pool": TEXT, "cpu_baseline": cpu, "cpu_baseline_threads": cpu,
           "repeats": {"n": 3, "values": [528513.2918336492] * 3, "min": 1.0, "median": 1.0, "max": 1.0},
           "noio": {"value": 728513.2918336492, "unit": bench.UNIT, "ms_per_step": 1.2, "kernel_ms_per_launch": 0.1, "roofline": roof}}
    w = wl.WORKLOADS[bench.HEADLINE[0]]
    names = [n if not m else f"{n} ({bench.mode_name(m)})" for n, m in bench.DEFAULT_SET]
    assert len(set(names)) == len(names)
    return {
        "metric": bench.METRIC, "value": 528513.2918336492, "unit": bench.UNIT, "n_gpus": 1, "steps": 20, "warmup": 5,
        "ms_per_step": 1.1805, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "int32", "data": "synthetic",
        "config": {"workload": bench.describe(w), "mode": "prefetch", "parallelism": "replicas x1 (independent requests per GPU)",
                   "l2": "flushed between steps (256 MiB write)", "host_pool": TEXT[:300], "graphs": "one CUDA graph per decode step"},
        "selected_entries_per_s": 1082395221.67, "gpu_launches": 3140, "roofline": roof, "noio": one["noio"], "e2e": e2e,
        "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap"], "samples": 61}, "headline": one,
        "per_workload": {n: one for n in names},
        "attention": {"kernel": "hs_mla_decode_kernel", "ms_per_launch": 0.0701234567, "frac": 0.2512345678, "bound": "hbm", "timing": TEXT,
                      "tensor": {"achieved": 260.1234567, "peak": 1908.5, "unit": "TFLOP/s", "frac": 0.136}},
        "run_s": 82.3456789, "cpu_baseline": cpu}


def test_the_printed_line_is_short_and_says_what_is_asked_of_it(capfd, monkeypatch):
    for name in ("RANK", "WORLD_SIZE", "LOCAL_RANK"):
        monkeypatch.delenv(name, raising=False)
    monkeypatch.setattr(bench, "Env", lambda *a: None)
    line = full_line()
    assert bench.run_gpu(types.SimpleNamespace(), lambda args, env: line) == 0
    out, err = capfd.readouterr()
    printed = [ln for ln in out.splitlines() if ln.startswith("{")]
    assert len(printed) == 1 and out.splitlines()[-1] == printed[0] and len(printed[0]) <= 2800
    got = json.loads(printed[0])
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
                "dtype", "data", "config", "clocks", "gpu_launches"):
        assert got[key] == line[key], key
    for key in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"):
        assert got["e2e"][key] == line["e2e"][key] or abs(got["e2e"][key] / line["e2e"][key] - 1) < 1e-7, key
    assert got["roofline"]["bound"] == "host_link" and abs(got["roofline"]["frac"] / line["roofline"]["frac"] - 1) < 1e-7
    assert got["cpu_baseline"]["kind"] == "oracle" and got["cpu_baseline"]["cores"] == 1
    assert set(got["per_workload"]) == set(line["per_workload"])
    assert all(abs(v / 528513.2918336492 - 1) < 1e-7 for v in got["per_workload"].values())
    full = [json.loads(ln) for ln in err.splitlines() if ln.startswith("{")]
    assert full == [line]


def test_a_longer_line_loses_its_extras_first():
    line = full_line()
    line["per_workload"] = {f"workload number {i} with a name": line["headline"] for i in range(100)}
    line["per_workload"]["broken"] = {"error": "RuntimeError: out of memory"}
    got = bench.brief(line)
    assert len(json.dumps(got)) <= 2800 and "per_workload" not in got
    assert got["value"] == line["value"] and got["e2e"]["h2d_bytes_per_step"] == 262144 and got["roofline"]["frac"] > 0
    line["per_workload"] = {"broken": {"error": "RuntimeError: " + "x" * 500}}
    assert bench.brief(line)["per_workload"]["broken"].startswith("RuntimeError")
