"""A refused call leaves nothing behind for the next one to trip over."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In a process of its own: a capture that was broken off leaves torch's random
# number generator waiting for its end.
PROGRAM = """
import torch
import sparse_communication_sharded_gb300 as pkg
from sparse_communication_sharded_gb300 import layers as L

params = torch.zeros(4096, device="cuda")
opt = pkg.Scape(params, 2, 0.9)
grads = [torch.ones(4096, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
torch.cuda.synchronize()
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(side):
    graph.capture_begin(capture_error_mode="thread_local")
    try:
        L.status()
        raise SystemExit("status() worked under capture")
    except pkg.ScapeError:
        pass
    try:
        graph.capture_end()
    except RuntimeError:
        pass  # the refused call ended the capture
opt.step(grads)
torch.cuda.synchronize()
assert bool(torch.isfinite(params).all()) and bool((params != 0).any())
opt.close()
print("stepped")
"""


def test_cuda_error_of_a_layer_call_is_not_the_optimizers(cuda_device):
    """status() has to synchronise, which a stream under capture refuses; the
    optimizer's next launches must not report that error as theirs."""
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "stepped" in r.stdout, r.stdout + r.stderr
