"""The line that bench.py prints: the headline whole, the rest summed up, short enough to survive a cut-off log."""

import json

import bench
from block_quantized_matmul_lwq_b200 import inputs


def record():
    call = {"M": 512, "N": 11008, "K": 4096, "ms": 0.12345, "GB/s": 1234.5, "path": "gemv"}
    names = ["q8_0_gemv_4096x4096", "q4_k_7b_layer_decode", "q4_k_7b_layer_decode_fused", "q4_0_gemv_11008x4096_act_i8",
             "q4_k_7b_layer_decode_act_i8", "q4_0_prefill_gemm", "q6_k_7b_layer_decode", "q5_k_7b_layer_decode",
             "q2_k_7b_layer_decode", "q6_k_prefill_gemm", "q5_k_prefill_gemm", "q2_k_prefill_gemm"]
    work = {n: {"steps": 4000, "ms_per_step": 0.12345, "launches_per_step": 14, "value": 1234.56, "unit": "TFLOP/s",
                "frac_of_bf16_sustained": 0.1234, "frac_of_bf16_peak": 0.1234, "per_call": [call] * 7,
                "clocks": {"sm_mhz": 1965.0, "sm_max_mhz": 1965.0, "power_w_max": 999.9, "reasons": ["sw_power_cap"],
                           "samples": 12}} for n in names}
    attention = {n: {"shape": {"B": 16, "H": 32, "Hkv": 32, "L": 4096, "D": 128, "dtype": "f16"}, "calls": 400,
                     "us_per_call": 165.12, "launches_per_call": 2, "bytes_per_call": 1073741824, "value": 6500.1,
                     "unit": "GB/s", "frac_of_hbm": 0.9911, "cache_copies": 2} for n in inputs.ATTENTION_WORKLOADS}
    points = [{"fmt": f, "M": M, "K": K, "N": N, "ms": 0.12345, "path": "gemv", "GB/s": 1234.5, "TFLOP/s": 123.45,
               "bound": "hbm", "frac": 0.001 * i} for i, (f, M, (K, N)) in enumerate(
                   (f, M, kn) for f in inputs.SWEEP_FMTS for M in inputs.SWEEP_MS for kn in inputs.SWEEP_SHAPES_KN)]
    text = "x" * 100
    return {"metric": bench.METRIC, "value": 2549.0, "unit": "GB/s", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": 0.030158, "config": {k: text for k in "abcdefgh"}, "roofline": {k: text for k in "abcdefghi"},
            "cpu_baseline": {"value": 2.78, "sample": text}, "e2e": {"value": 43.88, "unit": "GB/s"}, "gpu_launches": 60,
            "clocks": {"sm_mhz": 1965.0, "reasons": []}, "workloads": work, "attention": attention,
            "host_enqueue": {k: 1.2345 for k in "abcdefghij"}, "device_error": 0,
            "sweep": {"act": "f16", "peaks": {"hbm_gbs": 6545.0}, "frac": text, "points": points}}


def test_the_line_is_short_and_keeps_the_headline():
    full = record()
    line = bench.short_record(full)
    assert len(json.dumps(full)) > 16000 and len(json.dumps(line)) < 8000
    for key in set(full) - {"workloads", "attention", "sweep"}:
        assert line[key] == full[key]
    assert set(line["workloads"]) == set(full["workloads"]) and set(line["attention"]) == set(full["attention"])
    assert line["workloads"]["q4_k_7b_layer_decode"]["value"] == 1234.56
    assert line["sweep"]["points"] == len(full["sweep"]["points"]) and line["sweep"]["frac_least"] == 0.0
    assert full == record()                                       # (the record itself is left alone)


def test_what_was_left_out_stays_out():
    full = record()
    full["attention"] = full["sweep"] = None
    full["workloads"] = {}
    assert bench.short_record(full) == full
