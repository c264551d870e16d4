"""Products of 8-bit integers with scales far from one another: y = (sum * s_x) * s_w, so that no product of
two scales leaves fp32's range where y does not.

Sums are below 2^24 and exact; two products round once each, 2^-24 of their value or half of the
smallest subnormal, 2^-150: 4 u of y in all, and 2^-149.
"""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M

U = 2.0 ** -24


# integer dot products, tensor cores, tensor cores with K in pieces
@pytest.mark.gpu
@pytest.mark.parametrize("rows,K,N", [(5, 512, 100), (150, 1024, 300), (200, 512, 20000),
                                      (150, 4096, 2048)])
def test_scales_far_apart(rows, K, N):
    g = torch.Generator().manual_seed(rows + N)
    qx, qw = (torch.randint(-60, 61, s, generator=g, dtype=torch.int8).cuda()
              for s in ((rows, K), (1, N, K)))
    qx[3] = 0                                                 # sums of 0 under scales of 1e40
    sx = torch.rand(rows, generator=g) + 0.5
    sw = torch.rand(1, N, generator=g) + 0.5
    sx[0] *= 1e-30
    sx[3] *= 1e30
    sw[:, ::2] *= 1e-10
    sw[:, 1::4] *= 1e10
    sx, sw = sx.cuda(), sw.cuda()
    ws = M.alloc_int8_workspace(M.int8_matmul_workspace_size(rows, K, N, 1))
    y = torch.empty(rows, N, device="cuda")
    M.int8_matmul(qx, sx, qw, sw, None, y, ws)
    want = (qx.double() @ qw[0].double().T) * sx[:, None].double() * sw.double()
    assert M.device_status(ws) == 0
    assert ((y.double() - want).abs() <= 4 * U * want.abs() + 2.0 ** -149).all()
