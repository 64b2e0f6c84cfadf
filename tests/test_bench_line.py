"""The printed benchmark line stays short however much is measured: what reads it
may keep only the last few thousand characters of a program's output."""
import json

import pytest

import bench

pytestmark = pytest.mark.cpu

KEYS = ["metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
        "vs_baseline", "dtype", "data", "config", "roofline", "cpu_baseline", "e2e", "gpu_launches", "clocks"]


def record(name):
    x = 1234.567890123456
    roof = dict(bound="tensor", achieved=x, peak=3792.4, unit="TFLOP/s", frac=0.6722571417993809, flops=2886218022912.0,
                algorithmic_bytes=3861291008, t_compute_us=x, t_mem_us=x, traffic=1964497280.0,
                traffic_per_step=3928994560, algorithmic_bytes_per_launch=1930645504.0, launches_per_step=2,
                peak_source="measured bf16 burst x2")
    tactics = [{f"key_of_a_gemm_{i}": x for i in range(10)}] * 2
    cpu = dict(value=x, unit="TFLOP/s", cores=16, kind="oracle", sample="experts " + str(list(range(41))))
    return dict(value=x, unit="TFLOP/s", ms_per_step=x, ms_mean=x, per_gemm_ms=[x, x], useful_flops=x,
                config=bench.Workload(name).config(), l2=bench.L2_NOTE, roofline=roof, tactics=tactics, cpu_baseline=cpu)


def test_line_is_short_and_whole():
    head = record(bench.HEADLINE)
    full = {k: head.get(k, 1234.567890123456) for k in KEYS}
    full.update(metric=bench.METRIC, unit="TFLOP/s", data="synthetic", dtype="e4m3", scaling="weak",
                tactics=head["tactics"], per_gemm_ms=head["per_gemm_ms"], clocks=dict(
                    sm_mhz=2070.0, sm_max_mhz=2070.0, power_w_max=1235.35, reasons=[], samples=16, samples_under_load=9,
                    window="soak of the same steps + timed region", soak_s=1.0, timed_s=0.009),
                e2e=dict(value=1234.567890123456, unit="TFLOP/s", h2d_bytes_per_step=336448768, steps=20,
                         d2h_bytes_per_step=816054272, ms_per_step=1234.567890123456, pipelining="x" * 150),
                configs={name: record(name) for name in bench.CONFIGS})
    assert len(json.dumps(full)) > 12000
    line = bench.short_line(full)
    assert len(json.dumps(line)) <= 3000
    assert all(line[k] == full[k] for k in KEYS)
    assert list(line["configs"]) == bench.CONFIGS
    for name, r in line["configs"].items():
        assert r["ms_per_step"] == pytest.approx(full["configs"][name]["ms_per_step"], rel=1e-6)
        assert r["frac"] == pytest.approx(0.6722571, abs=1e-4)
    alone = {k: v for k, v in full.items() if k != "configs"}
    assert "configs" not in bench.short_line(alone)
