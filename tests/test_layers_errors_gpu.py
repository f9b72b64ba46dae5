"""A refused call leaves nothing behind for the next one to trip over."""
import pytest
import torch

import sparse_communication_sharded_gb300 as pkg
from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu


def test_cuda_error_of_a_layer_call_is_not_the_optimizers(cuda_device):
    """status() has to synchronise, which a stream under capture refuses; the
    optimizer's next launches must not report that error as theirs."""
    params = torch.zeros(4096, device="cuda")
    opt = pkg.Scape(params, 2, 0.9)
    grads = [torch.ones(4096, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin(capture_error_mode="thread_local")
        with pytest.raises(pkg.ScapeError):
            L.status()
        try:
            graph.capture_end()
        except RuntimeError:
            pass  # the refused call ended the capture
    opt.step(grads)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(params).all()) and bool((params != 0).any())
    opt.close()
