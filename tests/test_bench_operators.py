"""bench.py --operators: an unknown case is refused on the host (CPU), and a small case prints its line (GPU)."""
import json

import pytest

from test_bench_cli import run_bench


def test_an_unknown_case_is_refused():
    r = run_bench("--operators", "no such case")
    assert r.returncode == 2 and "no such case" in r.stderr


@pytest.mark.gpu
def test_one_case_prints_its_line():
    r = run_bench("--operators", "route decode", "--steps", "3")
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["mode"] == "operators" and [row["case"] for row in line["rows"]] == ["route decode"]
    assert line["rows"][0]["us"] > 0
