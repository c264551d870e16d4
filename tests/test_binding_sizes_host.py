"""Sizes that the library's 32-bit arguments do not hold: the binding refuses them, as they would reach the library as
other numbers (2^32 rows as none, 2^32 + 8 channels as eight) and the call would succeed without its work. Meta
tensors that say they are on a GPU, and a recorder in the library's place."""
import pytest
import torch

import sparse_moe_layer_route_gb300 as M
from test_binding_checks_host import OnGpu, calls  # noqa: F401

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


class Meta(OnGpu):
    def data_ptr(self):
        return 4096


def meta(*shape, dtype=BF16):
    return Meta(torch.empty(*shape, dtype=dtype, device="meta"))


def drop(T, d, residual=False, p=0.5):
    rng = meta(2, dtype=torch.int64)
    M.dropout(meta(T, d), p, rng, meta(T, d), residual=meta(T, d) if residual else None, stream=0)


@pytest.mark.parametrize("T,d", [(2 ** 32, 64), (2 ** 32 + 3, 1), (2 ** 31, 8), (1, 2 ** 32 + 8), (1, 2 ** 31),
                                 (2, 2 ** 33)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(calls, T, d, residual):  # noqa: F811
    with pytest.raises(ValueError):
        drop(T, d, residual)
    assert calls == []


def test_dropout_s_largest_sizes_reach_the_library(calls):  # noqa: F811
    drop(2 ** 31 - 1, 1)
    drop(1, 2 ** 31 - 1)                 # which the library itself refuses
    assert [args[:2] for _, args in calls] == [(2 ** 31 - 1, 1), (1, 2 ** 31 - 1)]


BIG = 2 ** 32 + 16


def rows(T, d):
    M.quantize_rows(meta(T, d), meta(T, d, dtype=I8), meta(T, dtype=F32), stream=0)


def product(T, K, N, n):
    ws = Meta(torch.zeros(1 << 16, dtype=torch.uint8))
    M.int8_matmul(meta(T, K, dtype=I8), meta(T, dtype=F32), meta(n, N, K, dtype=I8), meta(n, N, dtype=F32),
                  meta(n + 1, dtype=torch.int32), meta(T, N), ws, stream=0)


@pytest.mark.parametrize("call", [
    lambda: rows(BIG, 64), lambda: rows(2 ** 32, 1), lambda: rows(1, BIG), lambda: rows(0, 2 ** 31),
    lambda: product(BIG, 16, 16, 1), lambda: product(4, BIG, 16, 1), lambda: product(4, 16, BIG, 1),
    lambda: product(4, 16, 16, BIG), lambda: M.int8_matmul_workspace_size(BIG, 16, 16, 1),
    lambda: M.int8_matmul_workspace_size(4, BIG, 16, 1), lambda: M.int8_matmul_workspace_size(4, 16, BIG, 1),
    lambda: M.int8_matmul_workspace_size(4, 16, 16, BIG), lambda: M.quantize_channels(meta(BIG, 16, 16), stream=0),
    lambda: M.quantize_channels(meta(1, BIG, 16), stream=0), lambda: M.quantize_channels(meta(16, BIG), stream=0)])
def test_8_bit_entry_points(calls, call):  # noqa: F811
    with pytest.raises(ValueError):
        call()
    assert calls == []


def test_8_bit_sizes_below_reach_the_library(calls):  # noqa: F811
    rows(2 ** 31 - 1, 1)
    product(2 ** 31 - 1, 16, 16, 1)
    assert [args[0] for _, args in calls] == [2 ** 31 - 1] * 2
