"""What bench.py prints: one line on stdout that a reader of a pipe gets whole."""
import json
import sys

import bench


def test_the_line_on_stdout_is_short(monkeypatch, capsys):
    """One JSON line with the headline and the workloads' summary; their details, many KB, go to stderr."""
    workloads = {f"workload_{i}": {"us_per_call": float(i), "roofline": {"how": "x" * 300}} for i in range(40)}
    line = {"metric": bench.METRIC, "value": 1.5, "unit": bench.UNIT, "workloads": workloads, "workloads_summary": {"cols": ["us_per_call"]}}
    monkeypatch.setattr(bench, "run_ours", lambda args, dist: dict(line))
    monkeypatch.setattr(sys, "argv", ["bench.py"])
    bench.main()
    got = capsys.readouterr()
    assert len(got.out) < 8192 and got.out.count("\n") == 1
    assert json.loads(got.out) == {k: v for k, v in line.items() if k != "workloads"}
    assert json.loads(got.err.strip().splitlines()[-1]) == {"workloads": workloads}
