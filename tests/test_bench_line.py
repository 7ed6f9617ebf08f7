"""The line that bench.py prints to stdout: the contract's keys, and short however many workloads
and kernels a run has."""
import json

import bench

KEYS = ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better",
        "scaling", "vs_baseline", "dtype", "data", "config", "e2e", "gpu_launches", "clocks",
        "roofline", "cpu_baseline")


def record(workloads):
    kernels = {f"kernel {i}": {"bytes": 1e9, "hbm": {"frac": 0.123456789012345}, "what": "x" * 800}
               for i in range(6)}
    entry = {"workload": "w", "forward": "f", "tokens_per_s": 1.5, "ms_per_step": 2.5,
             "steps_ms": {"f": 2.5, "g": 3.5}, "kernels": kernels}
    out = {k: k for k in KEYS}
    out.update(headline=entry, configs={f"workload {i}": entry for i in range(workloads)},
               fma_peak={"tflops": 80.0, "runs": list(range(1000))},
               train={"metric": "m", "value": 3.0, "unit": "tokens/s", "ms_per_step": 4.0,
                      "kernels_ms": {"a": 1.0}, "roofline": kernels,
                      "stack": {"ours": {"ms_per_step": 5.0}, "dense_context": kernels}})
    return out


def test_line_is_short_and_whole():
    out = record(7)
    line = bench.brief(out)
    assert all(line[k] == out[k] for k in KEYS)
    assert len(json.dumps(out)) > 30000 and len(json.dumps(line)) < 4000
    assert line["configs"]["workload 3"] == {"forward": "f", "tokens_per_s": 1.5, "ms_per_step": 2.5}
    assert line["steps_ms"] == {"f": 2.5, "g": 3.5} and line["fma_peak"] == {"tflops": 80.0}
    assert line["train"]["ms_per_step"] == 4.0 and line["train"]["stack_ms"] == 5.0
    assert "headline" in out and "kernels" in out["configs"]["workload 0"]   # as it was


def test_line_of_a_run_without_the_parts():
    out = record(0)
    for k in ("train", "headline", "fma_peak", "configs"):
        del out[k]
    assert bench.brief(out) == out
