"""How much the gradient of the norms asks for: partial sums of the runs of tokens that can be under way, not of more."""
import pytest

import sparse_moe_layer_route_gb300 as M
from test_norm_host import lib  # noqa: F401


@pytest.mark.parametrize("d,per_sm,cluster", [
    (1, 2, 1), (256, 2, 1), (1024, 2, 1), (1025, 3, 1), (1280, 3, 1), (1281, 2, 1), (2048, 2, 1), (2049, 1, 1),
    (4096, 1, 1), (8192, 1, 1), (8193, 1, 2), (16384, 1, 2), (16385, 1, 4), (32768, 1, 4), (32769, 1, 8), (65536, 1, 8)])
def test_size_by_width(lib, d, per_sm, cluster):  # noqa: F811
    for T in (1, 7, 100, 152, 304, 5000, 2 ** 31 - 1):
        n = M.residual_norm_workspace_size(M.ResidualNormConfig.make(T, d))
        # six rows of fp32 sums for each run, of which a GPU has at least 152 SMs' and at most 160's
        runs = [min(T, per_sm * sms // cluster) for sms in (152, 160)]
        assert 24 * d * runs[0] <= n <= 24 * d * runs[1] + 255, T
