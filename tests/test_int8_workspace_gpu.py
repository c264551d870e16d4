"""One workspace for every number of rows up to the one that it was made for, whatever the earlier calls
left in it. Codes are at most 60 in magnitude and scales 1: outputs are exact sums."""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M


@pytest.mark.gpu
@pytest.mark.parametrize("K,N,n,most", [(2048, 2048, 1, 2048), (4096, 300, 7, 3000)])
def test_fewer_rows_in_a_workspace_for_more(K, N, n, most):
    g = torch.Generator().manual_seed(K)
    qx, qw = (torch.randint(-60, 61, s, generator=g, dtype=torch.int8).cuda()
              for s in ((most, K), (n, N, K)))
    ones = torch.ones(most, device="cuda")
    sw = torch.ones(n, N, device="cuda")
    ws = M.alloc_int8_workspace(M.int8_matmul_workspace_size(most, K, N, n))
    for rows in (most, 576, 97, 541, 192, 24, 1, 0, 1000):
        off = [rows * e // n for e in range(n + 1)]
        y = torch.full((rows, N), float("nan"), device="cuda")
        M.int8_matmul(qx[:rows], ones[:rows], qw, sw,
                      torch.tensor(off, dtype=torch.int32, device="cuda") if n > 1 else None, y, ws)
        for e in range(n):
            r = slice(off[e], off[e + 1])
            assert torch.equal(y[r].double(), qx[r].double() @ qw[e].double().T), (rows, e)
    assert M.device_status(ws) == 0
