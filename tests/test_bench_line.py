"""The benchmark's last line: one JSON object with what its readers need, short enough for one that keeps the last 8000
characters of the output."""
import importlib.util
import json
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bench():
    spec = importlib.util.spec_from_file_location("bench", os.path.join(ROOT, "bench.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def record(workloads):
    """A record as long as a full run's, and longer."""
    measured = {"shape": [14336, 4096], "M": 1, "gbps": 4635.6, "frac_hbm_peak": 0.5795, "weight_gbps": 4633.2, "mean_launch_us": 13.466,
                "replicas": 35, "weights_per_s": 4360686502536.6, "bytes_per_launch": 62422784}
    step = {f"gguf:q{i}_k": dict(measured, tensors=46) for i in range(5)}
    ceiling = {"gbps": 5600.1, "configurations": [dict(measured) for _ in range(8)]}
    return {"metric": "decode GB/s (payload+output) per format & % of HBM peak, 1×MI355X", "value": 5520.2, "unit": "GB/s", "n_gpus": 1,
            "steps": 20, "warmup": 5, "ms_per_step": 3.8459, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f32",
            "data": "synthetic", "config": {"workload": "w" * 80, **{f"figure_{i}": 1234.5678 for i in range(20)}},
            "roofline": {"bound": "hbm", "achieved": 6203.9, "peak": 8000.0, "frac": 0.7755, "copy_ceiling": ceiling, "frac_of_copy_ceiling": 1.07},
            "cpu_baseline": {"value": 0.4467, "sample": "s" * 130, "cpu_model": "c" * 40},
            "per_format": {"step": step, "ceilings": {f"ceiling {i} -> bf16": dict(ceiling) for i in range(6)},
                           "workloads": {**{f"all_formats gguf:iq{i}_xxs[14336, 4096]->bf16": dict(measured) for i in range(28)},
                                         **{f"gemm_q8_1 gguf:q4_k[14336, 4096] M={i}": {"tops": 341.8} for i in range(workloads)}}}}


def test_the_line_is_short_and_whole():
    b = bench()
    for workloads in (0, 80, 400):
        full = record(workloads)
        line = b.short_line(full)
        text = json.dumps(line)
        assert len(text) <= b.LINE_CHARS < 8000 and "\n" not in text
        for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline", "dtype",
                    "data", "config", "cpu_baseline"):
            assert line[key] == full[key]
        assert line["per_format"]["step"] == full["per_format"]["step"]
        assert line["roofline"]["copy_ceiling_gbps"] == 5600.1 and "copy_ceiling" in full["roofline"]
        assert len([k for k in line["per_format"]["workloads_gbps"] if k.startswith("all_formats")]) == 28
    assert len(json.dumps(record(80))) > 20000
    assert all(v == 341.8 for k, v in b.short_line(record(10))["per_format"]["workloads_gbps"].items() if k.startswith("gemm"))
