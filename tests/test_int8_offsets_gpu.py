"""Offsets that descend or leave [0, rows]: the segments they bound are empty and reported, every other
one is computed, on each path of the 8-bit products.

Codes are at most 60 in magnitude and K at most 4096, so sums stay below 2^24 and are exact; scales are
1, so outputs are those sums: compared for equality.
"""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M


def owners(off, rows):
    """The segment of each row (-1: none): the first sound one that holds it."""
    own = [-1] * rows
    for e in reversed(range(len(off) - 1)):
        if 0 <= off[e] <= off[e + 1] <= rows:
            own[off[e]:off[e + 1]] = [e] * (off[e + 1] - off[e])
    return torch.tensor(own)


def check(rows, K, N, off):
    g, n = torch.Generator().manual_seed(rows + K), len(off) - 1
    qx, qw = (torch.randint(-60, 61, s, generator=g, dtype=torch.int8).cuda()
              for s in ((rows, K), (n, N, K)))
    ws = M.alloc_int8_workspace(M.int8_matmul_workspace_size(rows, K, N, n))
    y = torch.full((rows, N), float("nan"), device="cuda")
    M.int8_matmul(qx, torch.ones(rows, device="cuda"), qw, torch.ones(n, N, device="cuda"),
                  torch.tensor(off, dtype=torch.int32, device="cuda"), y, ws)
    assert M.device_status(ws) == M.DEVFAULT_BAD_TILE
    own = owners(off, rows)
    for e in range(-1, n):
        r = torch.nonzero(own == e)[:, 0].cuda()
        if e < 0:
            assert torch.isnan(y[r]).all()
        else:
            assert torch.equal(y[r].double(), qx[r].double() @ qw[e].double().T), e


# three paths: integer dot products, tensor cores, tensor cores with K in pieces
@pytest.mark.gpu
@pytest.mark.parametrize("off", [[0, 500, 50, 150], [0, 30, 200, 40, 150], [-7, 20, 90, 150],
                                 [0, 60, 140, 151], [0, 150, -1, 0]])
@pytest.mark.parametrize("K,N", [(4096, 2048), (64, 300), (4096, 6500)])
def test_sound_segments_among_unsound_ones(off, K, N):
    check(150, K, N, off)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,at,value", [(1, 64, 50, -3), (1, 64, 63, 9), (3, 256, 256, 2),
                                             (8, 33, 32, 9), (300, 200, 150, 301)])
def test_unsound_segments_far_behind_the_rows_are_reported(rows, n, at, value):
    """All rows in the first segment, and a bad offset among many segments without a row."""
    off = [0] + [rows] * n
    off[at] = value
    check(rows, 64, 100, off)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,off", [
    (20, [0, 19, 0, 20]), (20, [8, 16, 0, 20, 4, 12]), (1500, [0, 1400, 0, 1500]),
    (1500, [700, 900, 100, 1500, 0, 1300])])
@pytest.mark.parametrize("K,N", [(64, 64), (3008, 600), (336, 5300)])
def test_rows_of_two_segments_have_the_first_ones_product(rows, off, K, N):
    """Sound segments between which offsets descend may share rows, and together hold more tiles than any
    that ascend."""
    check(rows, K, N, off)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,f", [(8, 128, 64), (600, 512, 384)])
@pytest.mark.parametrize("last", [lambda off: off[-2] - 3, lambda off: off[-3] - 1, lambda off: -1,
                                  lambda off: off[-1] + 10])
def test_experts_whose_last_offset_does_not_hold_them(T, d, f, last):
    """Positions past the last offset have no rows (they are those of dropped slots): an expert that
    reaches past it is empty and reported, and nothing is computed from what the workspace holds there."""
    E, k, g = 6, 2, torch.Generator().manual_seed(T)

    def w(K, N):
        return M.quantize_channels((torch.randn(E, K, N, generator=g) / K ** 0.5).bfloat16().cuda())

    cfg = M.MoeConfig.make(T, d, E, k, f)
    weights = M.make_int8_weights(w(d, f), w(d, f), w(f, d))
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    off = [T * k * e // E for e in range(E + 1)]
    perm = torch.randperm(T * k, generator=g).int().cuda()
    ws = M.alloc_int8_workspace(M.grouped_ffn_int8_workspace_size(cfg))
    outs = []
    for offsets in (off, off[:-1] + [last(off)]):
        y = torch.full((T * k, d), float("nan"), dtype=torch.float16, device="cuda")
        M.grouped_ffn_int8(cfg, x, perm, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                           None, weights, y, ws)
        outs.append((y, M.device_status(ws)))
        x = -2 * x                # what the workspace holds of the first call is not the second one's
    (first, status), (y, bad) = outs
    assert status == 0 and bad == M.DEVFAULT_BAD_TILE and not torch.isnan(first).any()
    x = x / 4
    whole = torch.empty_like(y)
    M.grouped_ffn_int8(cfg, -2 * x, perm, torch.tensor(off, dtype=torch.int32, device="cuda"), None,
                       weights, whole, ws)
    end = min(offsets[-1], T * k)
    for e in range(E):
        slot = perm[off[e]:off[e + 1]].long()
        sound = offsets[e] <= offsets[e + 1] <= T * k and offsets[e + 1] <= end
        if sound:
            assert torch.equal(y[slot], whole[slot]), e
        else:
            assert torch.isnan(y[slot]).all(), e
