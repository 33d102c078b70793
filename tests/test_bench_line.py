"""bench.py's line of standard output: every field that a reader needs, and short enough
that the end of a captured output holds it whole."""
import json

import bench

LEG = {"tokens": 64, "ms_per_step": 0.2902639389038086, "tokens_per_s": 220488.98062121714,
       "distinct_experts": 125.95, "kernel_ms": {k: 0.17172874882817268 for k in bench.SEGMENTS},
       "weights": "a description of the weights of this leg, " * 3,
       "step_hbm_frac": 0.5843443446991297}


def record():
    quant = {f: dict(LEG) for f in ("int8", "fp8", "mxfp4")}
    native = {f: {t: dict(LEG) for t in ("1", "8", "64", "256", "4096_skewed")}
              for f in ("fp8", "mxfp4")}
    return {
        "metric": bench.METRIC, "value": 220488.98062121714, "unit": "tokens/s", "n_gpus": 1,
        "steps": 20, "warmup": 5, "clock_warmup": {"seconds": 1.0}, "ms_per_step": 0.29026,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
        "data": "synthetic", "config": {"workload": "w" * 60, **{f"k{i}": i for i in range(10)}},
        "roofline": {f"key_{i}": 0.9328884499079517 for i in range(10)},
        "cpu_baseline": {f"key_{i}": "some words about it" for i in range(12)},
        "achievable": {f"key_{i}": 6263.817981204366 for i in range(8)},
        "gpu_clock_power": {"samples": [[i, 2.35] for i in range(400)]},
        "decode": {t: dict(LEG) for t in ("1", "8", "32", "64", "128", "256")},
        "prefill": dict(LEG), "dense_masked_ablation": {"64": dict(LEG), "4096": dict(LEG)},
        "quantized_experts_decode": quant, "quantized_experts_native_decode": native,
        "quantized_experts_prefill": quant, "tiny_f32": dict(LEG), "block": dict(LEG),
        "block_decode_quantized": {**quant, "bf16": dict(LEG)},
        "stack": {"layers": 30, "decode": dict(LEG), "prefill": {"ms": 51.5, "tokens_per_s": 1.6e5},
                  "decode_int8": dict(LEG)},
        "cpu_oracle_other_configs": {"decode_single_thread": {"tokens_per_s": 45.8}},
    }


def test_fields():
    r = record()
    line = json.loads(json.dumps(bench.short_line(r)))
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step",
              "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "config", "roofline",
              "cpu_baseline", "achievable"):
        assert line[k] == r[k], k
    legs = line["legs"]
    assert legs["decode"]["8"] == {"ms_per_step": 0.29026, "tokens_per_s": 220490.0}
    assert legs["prefill"]["ms_per_step"] == 0.29026
    assert legs["quantized_experts_native_decode"]["fp8"]["4096_skewed"]["tokens_per_s"] == 220490.0
    assert legs["stack"]["prefill"] == {"ms": 51.5, "tokens_per_s": 1.6e5}
    assert "gpu_clock_power" not in legs and "cpu_oracle_other_configs" not in legs


def test_length():
    assert len(json.dumps(record())) > 15000
    assert len(json.dumps(bench.short_line(record()))) < 6000


def test_legs_left_out():
    r = record()
    for k in ("prefill", "block", "stack", "dense_masked_ablation", "cpu_baseline"):
        r[k] = None
    line = bench.short_line(r)
    assert "prefill" not in line["legs"] and line["cpu_baseline"] is None
