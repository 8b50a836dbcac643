"""efla_get_status reads a device word a kernel file.  A process pays for the files it uses."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import time, torch
import exact_flow_recurrence_gb300 as efla

def median():
    t = []
    for _ in range(300):
        a = time.perf_counter()
        efla.efla_get_status()
        t.append(time.perf_counter() - a)
    return sorted(t)[150]

x = torch.zeros(1, 1, 1, 16, device="cuda")
median()
before = median()
s = torch.zeros(1, 1, 1, device="cuda")
efla.efla_gated_fwd(x, x, x, s, s)
efla.efla_gated_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], s[:, :, 0], s[:, :, 0], torch.zeros(1, 1, 16, 16, device="cuda"))
efla.efla_norm_fwd(x[0, 0], torch.ones(16, device="cuda"))
median()
print("COST", before, median())
"""


@pytest.mark.gpu
def test_status_reads_what_was_launched():
    """Five words before the gated rule, its step and the norm are used, nine after: 5/9 of the time, 0.8 with room."""
    env = dict(os.environ, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, cwd=ROOT, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    before, after = (float(x) for x in r.stdout.split("COST")[1].split())
    assert before < 0.8 * after, (before, after)
