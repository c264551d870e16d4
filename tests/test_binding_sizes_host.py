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
