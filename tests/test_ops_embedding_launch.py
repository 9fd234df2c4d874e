"""The embedding's gradient on both sides of the shared memory that a launch
gets without asking: 48 KB, which the sort's counters of V / 152 rows pass
between V = 54720 and V = 54721."""
import subprocess
import sys
from pathlib import Path

import pytest

from gpu_util import dev  # noqa: F401

ROOT = Path(__file__).resolve().parent.parent

# In a process of its own, smallest table first: a larger one asks for more
# shared memory, which every later launch in the process then has too.
SCRIPT = """
import torch
from weight_communication_gb300 import embedding
dev = torch.device("cuda:0")
g = torch.Generator(device=dev)
g.manual_seed(5)
for V in (54720, 54721, 54800, 54872, 54873):
    for id_type in (torch.int32, torch.int64):
        ids = torch.randint(0, V, (500,), generator=g, device=dev).to(id_type)
        ids[:3] = torch.tensor([0, V - 1, V - 1], device=dev)
        dy = torch.randint(-8, 9, (500, 8), generator=g, device=dev).float()    # sums are exact
        want = torch.zeros(V, 8, device=dev).index_add_(0, ids, dy)
        got = embedding.grad(dy, ids, V)
        assert torch.equal(got, want), (V, id_type)
        embedding.grad(dy, ids, V, out=got, accumulate=True)
        assert torch.equal(got, 2 * want), (V, id_type)
print("done")
"""


@pytest.mark.gpu
def test_tables_around_48_kb_of_counters(dev):
    run = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "done", run.stdout + run.stderr
