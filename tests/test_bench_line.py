"""The result line of bench.py: one short line on standard output, everything
measured beside it."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def bench():
    sys.path.insert(0, ROOT)
    import bench
    return bench


def _line():
    kernel = {"name": "k", "ms": 0.123456789012345, "note": "x" * 60}
    return {
        "metric": "m", "value": 144750193.08457848, "unit": "tokens/s", "n_gpus": 1, "steps": 20, "warmup": 5,
        "ms_per_step": 3.6220193481445313, "higher_is_better": True, "scaling": "weak", "vs_baseline": 9.8,
        "dtype": "fp8", "data": "synthetic", "config": {"workload": "w"}, "gpu_launches": 2000,
        "input_sha256": {str(i): "0" * 64 for i in range(12)},
        "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": []},
        "e2e": {"value": 2.07e7, "unit": "tokens/s", "h2d_bytes_per_step": 1, "d2h_bytes_per_step": 2},
        "step_ms_groups": {"median": 1.0, "groups": [1.23456789] * 500},
        "roofline": {"frac": 0.88, "per_instantiation": [kernel] * 100},
        "workloads": {"mlp": {"ms_per_step": 1.23456789, "per_instantiation": [kernel] * 200},
                      "only_parts": {"a": {"us": 1.0}}}}


def test_short_line_and_everything_beside_it(bench, capsys, tmp_path):
    line = _line()
    assert len(json.dumps(line)) > 30000
    bench.report(line)
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) < 3000
    got = json.loads(out)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
              "vs_baseline", "dtype", "data", "config", "gpu_launches", "clocks", "e2e"):
        assert k in got
    assert got["value"] == line["value"] and got["ms_per_step"] == line["ms_per_step"]
    assert got["e2e"] == line["e2e"] and got["clocks"] == line["clocks"]
    assert got["workloads"] == {"mlp": {"ms_per_step": 1.23457}}
    assert json.loads(err) == line
    path = tmp_path / "all.json"
    bench.report(line, str(path))
    out2, err = capsys.readouterr()
    assert out2 == out and err == "" and json.loads(path.read_text()) == line
