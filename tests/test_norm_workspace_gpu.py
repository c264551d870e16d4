"""The gradient of the norms stays inside the workspace that it asks for, and fills what it adds up."""
import pytest
import torch

import norm_reference as R
import sparse_moe_layer_route_gb300 as M
from test_norm_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(5000, 64), (5000, 300), (3000, 1000), (2000, 1100), (2000, 1900), (1000, 2050),
                                 (1000, 3900), (700, 8000), (400, 8200), (300, 20000), (200, 40000), (3, 40000), (1, 64)])
def test_what_lies_around_it_stays(T, d):
    c = Case(T, d, R.RMS, R.LAYER, gate=max(1, T // 7), bias=True)
    size = M.residual_norm_workspace_size(c.cfg)
    buf = torch.full((size + 2 * 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    inside = buf[65536:65536 + size]
    h_out = c.stream()
    got = c.gradients(h_out, c.d_h_out, c.d_n, inside)
    inside.fill_(255)
    again = c.gradients(h_out, c.d_h_out, c.d_n, inside)
    for name, v in got.items():
        assert torch.equal(v, again[name]), name
    assert (buf[:65536] == 0x5A).all() and (buf[65536 + size:] == 0x5A).all()
