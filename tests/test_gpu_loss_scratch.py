"""Workspaces that the binding makes for a call on another stream than the current one."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
N = 24 << 20  # (a block of its own, which the allocator hands out again as it is)


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_a_side_stream_gets_no_memory_that_the_current_stream_still_uses(how):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(N, dtype=torch.uint8, device=DEV)
    at = t.data_ptr()
    torch.cuda._sleep(200_000_000)  # about 0.1 s; then the current stream writes to t
    t.fill_(1)
    del t
    ws = kfac._scratch(N, DEV, None, side if how == "stream" else side.cuda_stream)
    assert ws.data_ptr() != at and ws.numel() >= N
    torch.cuda.synchronize()


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_dropped_while_the_side_stream_uses_it(how):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ws = kfac._scratch(N, DEV, None, side if how == "stream" else side.cuda_stream)
    at = ws.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    del ws
    t = torch.empty(N, dtype=torch.uint8, device=DEV)  # the current stream's
    assert t.data_ptr() != at
    torch.cuda.synchronize()


def test_the_default_stream_by_its_handle():
    """Handle 0 is the default stream: its memory is the current stream's own here."""
    ws = kfac._scratch(N, DEV, None, 0)
    at = ws.data_ptr()
    del ws
    assert torch.empty(N, dtype=torch.uint8, device=DEV).data_ptr() == at


def test_dropped_while_the_current_stream_reads_the_error_word():
    side = torch.cuda.Stream()
    ws = kfac._scratch(N, DEV, None, side)
    at = ws.data_ptr()
    torch.cuda._sleep(200_000_000)
    flag = ws[:4].clone()
    del ws
    assert kfac._scratch(N, DEV, None, side).data_ptr() != at
    torch.cuda.synchronize()
    del flag
