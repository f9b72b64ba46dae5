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


def test_example_does_not_use_incomplete_gradients(cuda_device, monkeypatch):
    """A wait given up in a step's products ends training before the optimizer reads them."""
    from tests.test_layers_train_gpu import example
    steps = []
    monkeypatch.setattr(example.Scape, "step", lambda self, grads: steps.append(1))
    monkeypatch.setattr(example.Scape, "refresh_mask", lambda self: None)
    backward = example.Blocks.backward

    def backward_that_gives_up(*a):
        r = backward(*a)
        if len(steps) == 2:
            probe(1000)
        return r

    monkeypatch.setattr(example.Blocks, "backward", backward_that_gives_up)
    L.status()
    with pytest.raises(RuntimeError, match="incomplete"):
        example.train(workers=2, steps=5, hidden=64, blocks=1, tokens=32, out=8)
    assert len(steps) == 2
