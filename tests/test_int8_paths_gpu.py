"""8-bit products and experts on the tensor cores: rows of no segment, and segments of very uneven length.

Products: codes of at most 60 in magnitude and scales of 1, so sums are below 2^24 and outputs exact.
Experts: the tolerances of test_int8_gpu.py.
"""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M
from test_int8_gpu import check, experts64, layer


@pytest.mark.gpu
@pytest.mark.parametrize("counts,K,N", [
    ([90, 0, 60], 4096, 2048), ([33], 4096, 3001),                # K in pieces
    ([20] * 60, 1024, 700), ([100] * 16, 704, 520), ([1700, 0, 1, 300], 528, 1000),
    ([2000, 3, 0, 1] + [2] * 60, 1040, 520)])                     # a long segment among short ones
@pytest.mark.parametrize("before,after", [(0, 5), (7, 300)])
def test_rows_of_no_segment_are_left(counts, K, N, before, after):
    """Rows in front of the first offset and behind the last one."""
    n, rows = len(counts), before + sum(counts) + after
    assert rows > 8 and rows * K * N > 4e8                        # not the integer dot products'
    off = [before]
    for c in counts:
        off.append(off[-1] + c)
    g = torch.Generator().manual_seed(rows)
    qx, qw = (torch.randint(-60, 61, s, generator=g, dtype=torch.int8).cuda()
              for s in ((rows, K), (n, N, K)))
    ws = M.alloc_int8_workspace(M.int8_matmul_workspace_size(rows, K, N, n))
    y = torch.full((rows, N), float("nan"), device="cuda")
    M.int8_matmul(qx, torch.ones(rows, device="cuda"), qw, torch.ones(n, N, device="cuda"),
                  torch.tensor(off, dtype=torch.int32, device="cuda"), y, ws)
    assert M.device_status(ws) == 0
    assert torch.isnan(y[:before]).all() and torch.isnan(y[off[-1]:]).all()
    for e in range(n):
        r = slice(off[e], off[e + 1])
        assert torch.equal(y[r].double(), qx[r].double() @ qw[e].double().T), e


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,k,f,S", [(1500, 256, 64, 1, 256, 0), (700, 512, 64, 2, 320, 1),
                                         (3000, 192, 16, 2, 256, 0)])
def test_most_tokens_on_one_expert(T, d, E, k, f, S):
    """One segment of every token, whose tiles' height follows the mean of all."""
    assert T > 12 and 3 * T * (k + S) * d * f > 1e8               # not the integer dot products'
    cfg, st = layer(T, d, E, k, f, S, 0, seed=T, one_expert=True)
    assert (st["offsets"][2] - st["offsets"][1]).item() == T
    y = torch.full(((k + S) * T, d), float("nan"), dtype=torch.float16, device="cuda")
    M.grouped_ffn_int8(cfg, st["x"], st["perm_slot"], st["offsets"], st["topk_w"], st["weights"], y,
                       st["ws"])
    assert M.device_status(st["ws"]) == 0
    check(y, experts64(cfg, st))
