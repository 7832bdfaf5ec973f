"""The numbers of one bench.py line belong together."""

import json
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


def test_ratio_is_to_the_step_with_the_orthogonalised_step_timed_too():
    """--muon times another step between the headline and the comparison that divides by it."""
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--workload", "llama60m", "--steps", "3", "--warmup",
                        "1", "--muon", "--no-cpu-baseline"], capture_output=True, text=True, cwd=ROOT, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    wc = line["weight_centric"]
    assert line["muon_step"]["ms"] > 0
    assert wc["ratio_to_input_centric"] == pytest.approx(wc["ms_per_step"] / line["ms_per_step"], rel=1e-9)
