"""Tensors that an entry point allocates belong to the stream that it was given."""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_prepared_weights_on_another_stream(raw):
    """Memory that the current stream has freed, but still writes to, is not another stream's yet."""
    W = torch.randn(2, 512, 384, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q0, s0 = M.quantize_channels(W)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        late = torch.empty_like(q0), torch.empty_like(s0)
        torch.cuda._sleep(40_000_000)                # about 20 ms
        for t in late:
            t.fill_(77)
        del late, t
        q, s = M.quantize_channels(W, stream=side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        assert torch.equal(q, q0) and torch.equal(s, s0)
