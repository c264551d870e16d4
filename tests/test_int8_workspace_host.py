"""A workspace made for the largest number of rows serves every smaller one."""
import pytest

import sparse_moe_layer_route_gb300 as M
from sparse_moe_layer_route_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()


@pytest.mark.parametrize("K,N,n", [(2048, 2048, 1), (2048, 7168, 1), (4096, 4096, 1), (7168, 2048, 1),
                                   (16384, 250, 1), (4096, 300, 7), (4288, 1049, 3), (512, 512, 38),
                                   (65536, 16, 1), (1024, 1024, 20), (7168, 64, 64), (16, 1, 1)])
def test_product_workspaces_grow_with_the_rows(K, N, n):
    last = 0
    for rows in range(0, 6000):
        size = M.int8_matmul_workspace_size(rows, K, N, n)
        assert size >= last, rows
        last = size


@pytest.mark.parametrize("shared", [0, 2])
def test_expert_workspaces_grow_with_the_tokens(shared):
    last = 0
    for T in range(0, 3000):
        size = M.grouped_ffn_int8_workspace_size(M.MoeConfig.make(T, 512, 32, 4, 256, n_shared=shared))
        assert size >= last, T
        last = size


MOST = 2 ** 31 - 1
FAKE = 0x10000000  # never dereferenced


@pytest.mark.parametrize("size", [MOST, MOST - 255, MOST - 1022])
def test_sizes_near_the_end_of_32_bits_are_refused(size):
    """Sizes to which a tile or a block of threads cannot be added in 32 bits."""
    lib, n = M.lib(), M.ctypes.c_size_t(0)
    assert lib.moe_quantize_rows(1, size, 1, FAKE, 0, FAKE, FAKE, None) == 2
    assert lib.moe_quantize_channels(1, size, 1, FAKE, FAKE, FAKE, None) == 2
    assert lib.moe_quantize_channels(1, 1, size, FAKE, FAKE, FAKE, None) == 2
    assert lib.moe_int8_matmul_workspace_size(size, 16, 1, 1, M.ctypes.byref(n)) == 2
    assert lib.moe_int8_matmul(size, 16, 1, 1, FAKE, FAKE, FAKE, FAKE, None, 0, FAKE, FAKE, 1 << 40,
                               None) == 2
