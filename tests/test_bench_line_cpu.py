"""The bench's line: whole in a log's last few kilobytes, the contract's figures to their last digit."""
import json

import bench


def test_the_line_is_short_and_keeps_its_figures():
    third = 1e9 / 3
    times = {"fwd_ms": third, "bwd_wavefront_ms": third, "fwd_bwd_ms": third, "cells_per_s": third, "peak_MB": third, "peak_MB_above_inputs": third,
             "workspace_MB": third, "latency_floor_ms": third, "roofline": {k: third for k in ("hbm_us", "sfu_us", "bound_us", "frac")}}
    line = {"metric": bench.METRIC, "value": third, "unit": "cells/s", "n_gpus": 8, "steps": 100000, "warmup": 1000, "ms_per_step": third,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f32", "data": "synthetic",
            "config": {"workload": bench.WORKLOAD, "B": 32, "cells_per_step": 16777216, "launch": "x" * 60},
            "per_mode": {m: dict(times) for m in ("unfused", "fused", "unfused+extended", "fused+extended", "fused_checkpoint")},
            "roofline": {"bound": "hbm", "achieved": third, "peak": third, "unit": "GB/s", "frac": third, "traffic": 79181056, "kernel": "k" * 60,
                         "peak_source": "s" * 200, "latency": {"frac": third, "note": "n" * 200}},
            "per_config": {"sweep": [dict(times) for _ in range(60)]},
            "cpu_baseline": {"value": third, "unit": "cells/s", "cores": 16, "sample": "s" * 100, "single_core": {"value": third}},
            "e2e": {"value": third, "unit": "cells/s", "h2d_bytes_per_step": 16777472, "d2h_bytes_per_step": 16777472, "ms_per_step": third},
            "gpu_launches": 13000, "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": [], "samples": 5}, "wall_s_timed": third}
    text = json.dumps(bench.headline(line))
    assert len(text) <= 2600
    short = json.loads(text)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline", "dtype", "data",
                "config", "e2e", "gpu_launches", "clocks"):
        assert short[key] == line[key], key
    assert abs(short["per_mode"]["fused"]["fwd_bwd_ms"] / third - 1) < 1e-5 and short["roofline"]["bound"] == "hbm"
    assert "per_config" not in short and line["per_config"]["sweep"]      # what is left out is left in the whole
