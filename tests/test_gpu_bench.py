"""The benchmark's timed region holds its steps and nothing else."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_step_takes_what_its_launches_take():
    """The three convolutions' own times, measured launch by launch before the timed region, add up to a step's
    (within a factor of two: clocks and the gaps between launches differ); a full collection of the
    interpreter's objects inside the timed region would make a step four times as long."""
    steps = 50
    run = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--steps", str(steps), "--cpu-fraction", "0.01"],
                         cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert run.returncode == 0, run.stderr[-2000:]
    line = json.loads(run.stdout.strip().splitlines()[-1])
    launches = sum(w["us_mean"] for w in line["per_workload"].values())
    assert line["steps"] == steps and line["ms_per_step"] * 1e3 < 2 * launches
