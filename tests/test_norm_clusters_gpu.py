"""Norms around a block on rows that a cluster of CTAs shares (more than 8192 channels), many rows to a cluster: its
sums are exchanged row after row through the CTAs' shared memory, stages are refilled, and parameters' sums and rows
of gates go over the run of tokens that a cluster has."""
import pytest
import torch

import norm_reference as R
import sparse_moe_layer_route_gb300 as M
from test_norm_gpu import BF16, F16, F32, Case

pytestmark = pytest.mark.gpu


def run_of(T, d):
    """Tokens of a cluster in the gradient on a GPU of 152 SMs: clusters of 2, 4 or 8 CTAs, one an SM."""
    cl = 2
    while -(-(-(-d // 8)) // cl) * 8 > 8192:
        cl *= 2
    return -(-T // (152 // cl))


@pytest.mark.parametrize("T,d", [(1000, 8200), (1001, 8201), (700, 16384), (403, 16385), (300, 32768), (200, 65536),
                                 (150, 65535)])
@pytest.mark.parametrize("after,before,gates", [(R.RMS, R.RMS, "all"), (R.LAYER, R.LAYER, "third"),
                                                (R.NONE, R.RMS, "each"), (R.RMS, R.LAYER, "seven"),
                                                (R.LAYER, R.NONE, "none")])
def test_many_rows(T, d, after, before, gates):
    # sums over tokens: a cluster's run one after the other, then the clusters' within 32 + 16 adds
    assert 2 <= run_of(T, d) <= 80
    gate = {"all": T, "third": T // 3, "each": 1, "seven": 7, "none": 0}[gates]
    c = Case(T, d, after, before, gate=gate, bias=gates != "all", alpha=0.75, beta=1.25,
             p=0.1 if gates in ("third", "all") else 0.0)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("h,y,w", [(F32, F32, F32), (F32, BF16, BF16), (F16, F16, F32), (BF16, F32, F16)])
@pytest.mark.parametrize("T,d,pad", [(600, 12288, 0), (600, 12290, 3), (500, 16384, 8)])
def test_types_and_strides(T, d, pad, h, y, w):
    c = Case(T, d, R.LAYER, R.RMS, h=h, y=y, w=w, gate=100, bias=True, pad_h=pad, pad_y=2 * pad)
    c.check_forward()
    c.check_backward(c.d_h_out, c.d_n)


@pytest.mark.parametrize("d", [8200, 16385, 65536])
def test_calls_repeat_bit_for_bit(d):
    c = Case(400, d, R.RMS, R.LAYER, gate=90, bias=True, p=0.1)
    first, h_out = c.run(), c.stream()
    grads = c.gradients(h_out, c.d_h_out, c.d_n)
    for _ in range(10):
        for a, b in zip(first, c.run()):
            assert torch.equal(a, b)
        again = c.gradients(h_out, c.d_h_out, c.d_n)
        for name in grads:
            assert torch.equal(grads[name], again[name]), name


def test_in_place_and_in_a_graph():
    c = Case(300, 9000, R.RMS, R.RMS, gate=60)
    h_out, n = c.run()
    h, y = c.h.clone(), c.y.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        M.residual_norm(c.cfg, h, y, h, y, **c.w)
    for _ in range(3):
        h.copy_(c.h)
        y.copy_(c.y)
        graph.replay()
        assert torch.equal(h, h_out) and torch.equal(y, n)
