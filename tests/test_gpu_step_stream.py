"""The step's own buffers belong to the stream that a call is given."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac, workloads
from second_order_optimisation_gb300.step import KfacStep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_first_weight_gradients_on_another_stream(handle):
    """While the current stream is busy, a step on another one makes its gradients: nothing that waits on the
    current stream may write to them later."""
    layer = workloads.Layer("head", 256, 128, 1, 1, 0, 1, 1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, g = torch.randn(500, 256, device="cuda", generator=gen), torch.randn(500, 128, device="cuda", generator=gen)
    ca, cg = kfac.Checkpoint.empty(500, 256), kfac.Checkpoint.empty(500, 128)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, ca), kfac.CheckpointItem(g, cg)])
    want = KfacStep([layer], 500).weight_grads([ca], [cg])[0].clone()
    kf, side, busy = KfacStep([layer], 500), torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):  # some 5 ms
        busy = busy @ busy * 1e-2
    got = kf.weight_grads([ca], [cg], stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and bool(torch.count_nonzero(want))
