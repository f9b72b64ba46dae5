"""A wait that runs out is reported, once, and leaves the context usable."""
import pytest
import torch

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu


def probe(ns):
    assert C.load().scape_layer_probe_wait(ns, torch.cuda.current_stream().cuda_stream) == C.SCAPE_OK


def test_a_wait_that_runs_out(cuda_device):
    L.status()
    probe(1_000_000)
    assert L.status() == 1
    assert L.status() == 0
    probe(1)
    probe(1)
    assert L.status() == 2
    x, w = torch.ones(64, 128, device="cuda").bfloat16(), torch.ones(32, 128, device="cuda").bfloat16()
    assert bool((L.linear(x, w) == 128).all())
    assert L.status() == 0


def test_report_is_not_lost_to_another_stream(cuda_device):
    """Waits given up on one stream while another asks: every one is told of."""
    L.status()
    side = torch.cuda.Stream()
    told = 0
    for _ in range(8):
        with torch.cuda.stream(side):
            probe(1000)
        told += L.status()  # of this stream's work, and what else has been counted
    side.synchronize()
    assert told + L.status() == 8
