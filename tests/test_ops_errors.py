"""An error is reported by the call that met it, and by no later one."""
import subprocess
import sys
from pathlib import Path

import pytest

from gpu_util import dev  # noqa: F401

ROOT = Path(__file__).resolve().parent.parent

# The refusal: a launch on the default stream while a stream that waits for it is
# being captured, which CUDA answers with an error (and ends the capture).  In a
# process of its own, whose one capture fails.
SCRIPT = """
import ctypes
import torch
from weight_communication_gb300 import binding, embedding, fp8, gradnorm
dev = torch.device("cuda:0")
table = torch.randn(100, 64, device=dev)
ids = torch.arange(40, device=dev)
out = torch.empty(40, 64, device=dev)
dtable = torch.empty(100, 64, device=dev)
x = torch.full((1000,), 3.0, device=dev)
lists = [gradnorm.TensorList([x]), gradnorm.TensorList([torch.empty_like(x)])]
binding.calls()
torch.cuda.synchronize()

handle = ctypes.c_void_p()
assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))) == 0
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(torch.cuda.ExternalStream(handle.value, device=dev)):
    graph.capture_begin()
try:
    embedding.lookup(table, ids, out=out)
    raise SystemExit("a launch beside a capture was not refused")
except binding.WcError as e:
    assert e.code == binding.WC_ECUDA
with torch.cuda.stream(torch.cuda.ExternalStream(handle.value, device=dev)):
    try:
        graph.capture_end()
    except RuntimeError:
        pass
embedding.lookup(table, ids, out=out)
assert torch.equal(out, table[ids])
embedding.grad(out, ids, 100, out=dtable)
assert torch.equal(dtable[:40], table[:40]) and not bool(dtable[40:].any())
stats = gradnorm.clip(lists[0], 1.0, out=lists[1])
assert 0 < float(stats[1]) < 1 and float(lists[1].tensors[0][0]) == 3.0 * float(stats[1])
q, _ = fp8.quantize(torch.ones(5, 64, device=dev))
assert bool((fp8.matmul(q, q) == 64).all())
assert binding.wait_timeouts() == 0
print("done")
"""


@pytest.mark.gpu
def test_an_error_is_reported_once(dev):
    run = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "done", run.stdout + run.stderr
