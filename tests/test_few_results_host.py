"""Results of the few-token layer at addresses that are not a multiple of four are refused: the kernel would store whole
words there. On the CPU; no call gets as far as a launch."""
import ctypes

import pytest

import sparse_moe_layer_route_gb300 as M
from test_few_host import A, B, BASE, ROUTE, lib  # noqa: F401


@pytest.mark.parametrize("name", ROUTE)
@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("T", [0, 4])
def test_results_between_words(lib, name, off, T):  # noqa: F811
    cfg = M.MoeConfig.make(**{**BASE, "T": T})
    w = M.make_weights(A, A, A, A, A)
    r = M.make_route_out(**{name: B + off})
    ref = ctypes.byref
    assert lib.moe_layer_forward_few(ref(cfg), ref(w), A, None, B, ref(r), 0x100, 1 << 30, None) == 1
