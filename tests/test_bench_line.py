"""bench.py's stdout line: short enough to survive a reader that keeps the last
3000 characters, with the keys of the measurement in it."""
import copy
import json

import bench


def _record(workload):
    op = {"bound": "hbm", "achieved": 4901.683562584633, "peak": 6675.8, "unit": "GB/s", "frac": 0.7342466165230586,
          "peak_source": "hbm_gbs of measured peaks", "ms_per_launch": 6.444174337387085,
          "flop_per_launch": 7696581394432.0, "bytes_per_launch": 31587303424.0, "tflops": 1194.3471717980754,
          "gbs": 4901.683562584633, "t_tensor_ms": 2.010391127999164, "t_hbm_ms": 4.7316132035111895,
          "tensor_frac": 0.3119703196630642, "hbm_frac": 0.7342466165230586, "traffic": 31735763750.092796,
          "traffic_note": "x" * 160, "ms_x_sm_mhz": 12904.459110617638}
    return {"metric": bench.METRIC, "value": 658847.5687286888, "unit": "tokens/s", "n_gpus": 1, "steps": 20,
            "warmup": 5, "ms_per_step": 24.867664051055907, "higher_is_better": True, "scaling": "weak",
            "vs_baseline": None, "dtype": "mxfp8", "data": "synthetic",
            "config": {"workload": workload, "T": 16384, "H": 7168, "E": 256, "k": 8, "F": 2048, "S": 2048,
                       "score": "sigmoid", "pass": "fwd+bwd",
                       "l2": "flushed (512 MB write) before every timed step, outside the events",
                       "parallelism": "replicas x1", "cuda_graph": True},
            "expert_gemm_tflops_per_gpu": 1566.851764979411, "expert_gemm_frac_of_bf16_peak": 0.8185413044506379,
            "roofline": {**op, "kernel": "wgrad_fc1 grouped GEMM (tcgen05, mxf8f6f4 block-scaled)",
                         "why_this_kernel": "the longest grouped GEMM of the step, timed alone"},
            "gemm_ops": {f"op{i}": dict(op) for i in range(8)}, "experts_with_rows": 252,
            "stages_ms": {f"stage{i}": 0.14142719954252242 for i in range(8)},
            "e2e": {"value": 651225.7262291097, "unit": "tokens/s", "h2d_bytes_per_step": 469762048,
                    "d2h_bytes_per_step": 234881024, "how": "y" * 230},
            "gpu_launches": 620,
            "clocks": {"sm_mhz": 2002.5, "sm_max_mhz": 2070.0, "power_w_max": 1363.72, "reasons": ["sw_power_cap"],
                       "samples": 20, "samples_under_load": 18},
            "cpu_baseline": {"value": 0.9500256848944163, "unit": "tokens/s", "cores": 16, "kind": "oracle",
                             "sample": "z" * 170}}


def test_line_is_short_and_complete():
    out = _record("dsv3_mxfp8")
    out["configs"] = {name: _record(name) for name in bench.SUITE[:-1]}
    out["headline"] = "h" * 140
    before = copy.deepcopy(out)
    line = bench.summary(out)
    assert out == before                                    # (the complete record, for --details)
    text = json.dumps(line)
    assert len(text) <= 2600 and len(json.dumps(out)) > 20000
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "gpu_launches", "e2e", "clocks", "roofline", "cpu_baseline"):
        assert key in line, key
    assert line["value"] == out["value"] and line["ms_per_step"] == out["ms_per_step"]
    assert line["config"] == out["config"] and line["clocks"] == out["clocks"]
    for key in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"):
        assert key in line["e2e"]
    assert set(line["configs"]) == set(bench.SUITE[:-1])
    one = bench.summary(_record("tiny"))                    # a single workload
    assert "configs" not in one and "gemm_ops" not in one and len(json.dumps(one)) <= 2600
