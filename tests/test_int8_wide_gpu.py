"""Experts of more channels than 32-bit integer sums of 8-bit products hold (133 thousand of 127 * 127).

Tolerance: sums of K products on the tensor cores are within K / 16 * 2^-23 of the largest partial sum,
here the sum itself: 2e-3 at K = 262144; H's codes, the two scales and fp16 add under 1e-2: 2e-2.
"""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12])
def test_sums_past_32_bits(T):
    d, f = 262144, 64
    x = torch.ones(T, d, device="cuda").bfloat16()

    def w(K, N, value):
        return M.quantize_channels(torch.full((1, K, N), value, device="cuda").bfloat16())

    cfg = M.MoeConfig.make(T, d, 1, 1, f)
    weights = M.make_int8_weights(w(d, f, 2.0 ** -17), w(d, f, 2.0 ** -18), w(f, d, 2.0 ** -6))
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    y = torch.empty(T, d, dtype=torch.float16, device="cuda")
    ws = M.alloc_int8_workspace(M.grouped_ffn_int8_workspace_size(cfg))
    M.grouped_ffn_int8(cfg, x, perm, offsets, None, weights, y, ws)
    # g = 2, u = 1, h = 2 / (1 + exp(-2)) in 64 channels, each with weight 1 / 64
    want = 2 / (1 + torch.exp(torch.tensor(-2.0, dtype=torch.float64))).item()
    assert M.device_status(ws) == 0
    assert ((y.double() - want).abs() <= 2e-2 * want).all()
