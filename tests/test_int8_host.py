"""Argument checks of routing from logits and of the 8-bit entry points: every call below fails
before any launch, so no GPU is needed."""
import ctypes

import pytest

import sparse_moe_layer_route_gb300 as M
from sparse_moe_layer_route_gb300 import _build

FAKE = 0x10000000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return M.lib()


def gate(**kw):
    base = dict(T=4, E=16, top_k=2)
    base.update(kw)
    return M.GateConfig.make(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(top_k=0), 1), (dict(score=2), 1), (dict(score=-1), 1),
    (dict(dtype=3), 1), (dict(dtype=M.DTYPE_F16), 2), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(ld=15), 1), (dict(E=257), 2), (dict(top_k=9), 2),
    (dict(E=4, top_k=5), 2), (dict(n_groups=-1), 1), (dict(n_groups=3), 2),
    (dict(E=130, n_groups=65, topk_groups=1), 2), (dict(n_groups=4, topk_groups=0), 1),
    (dict(n_groups=4, topk_groups=5), 1), (dict(n_groups=8, topk_groups=1, top_k=3), 1),
])
def test_bad_gate_configs(lib, kw, status):
    c = gate(**kw)
    assert lib.moe_route_logits(ctypes.byref(c), FAKE, None, FAKE, FAKE, None, None) == status
    assert lib.moe_route_logits_backward(ctypes.byref(c), FAKE, FAKE, FAKE, None, FAKE,
                                         None) == status


def test_gate_pointers(lib):
    c = ctypes.byref(gate())
    assert lib.moe_route_logits(None, FAKE, None, FAKE, FAKE, None, None) == 1
    for a in ((None, None, FAKE, FAKE, None), (FAKE, None, None, FAKE, None),
              (FAKE, None, FAKE, None, None), (FAKE + 2, None, FAKE, FAKE, None),
              (FAKE, FAKE + 1, FAKE, FAKE, None), (FAKE, None, FAKE + 2, FAKE, None),
              (FAKE, None, FAKE, FAKE, FAKE + 1)):
        assert lib.moe_route_logits(c, *a, None) == 1
    for a in ((None, FAKE, FAKE, None, FAKE), (FAKE, None, FAKE, None, FAKE),
              (FAKE, FAKE, None, None, FAKE), (FAKE, FAKE, FAKE, None, None),
              (FAKE, FAKE, FAKE, FAKE + 2, FAKE), (FAKE, FAKE, FAKE, None, FAKE + 2)):
        assert lib.moe_route_logits_backward(c, *a, None) == 1
    # an empty batch examines no pointer
    e = ctypes.byref(gate(T=0))
    assert lib.moe_route_logits(e, None, None, None, None, None, None) == 0
    assert lib.moe_route_logits_backward(e, None, None, None, None, None, None) == 0


def test_quantize_arguments(lib):
    q = lib.moe_quantize_rows
    assert q(-1, 8, 0, FAKE, 0, FAKE, FAKE, None) == 1
    assert q(1, 0, 0, FAKE, 0, FAKE, FAKE, None) == 1
    assert q(1, 8, 3, FAKE, 0, FAKE, FAKE, None) == 1
    assert q(1, 8, 0, FAKE, 7, FAKE, FAKE, None) == 1
    assert q(1, 8, 0, FAKE + 2, 0, FAKE, FAKE, None) == 1
    assert q(1, 8, 1, FAKE + 1, 0, FAKE, FAKE, None) == 1
    assert q(1, 8, 0, None, 0, FAKE, FAKE, None) == 1
    assert q(1, 8, 0, FAKE, 0, None, FAKE, None) == 1
    assert q(1, 8, 0, FAKE, 0, FAKE, FAKE + 1, None) == 1
    assert q(0, 8, 0, None, 0, None, None, None) == 0
    c = lib.moe_quantize_channels
    assert c(0, 8, 8, FAKE, FAKE, FAKE, None) == 1
    assert c(1, 8, 8, None, FAKE, FAKE, None) == 1
    assert c(1, 8, 8, FAKE + 1, FAKE, FAKE, None) == 1
    assert c(70000, 8, 8, FAKE, FAKE, FAKE, None) == 2


@pytest.mark.parametrize("shape,status", [
    ((-1, 64, 8, 1), 1), ((4, 0, 8, 1), 1), ((4, 64, 0, 1), 1), ((4, 64, 8, 0), 1),
    ((4, 72, 8, 1), 2), ((4, 65552, 8, 1), 2), ((4, 64, 1 << 27, 1), 2), ((4, 64, 8, 257), 2),
    ((0, 64, 8, 1), 0), ((4, 64, 8, 256), 0)])
def test_matmul_shapes(lib, shape, status):
    n = ctypes.c_size_t(0)
    assert lib.moe_int8_matmul_workspace_size(*shape, ctypes.byref(n)) == status


def test_matmul_arguments(lib):
    need = M.int8_matmul_workspace_size(4, 64, 8, 2)

    def call(qx=FAKE, sx=FAKE, qw=FAKE, sw=FAKE, off=FAKE, dt=0, y=FAKE, ws=FAKE, n=need, rows=4):
        return lib.moe_int8_matmul(rows, 64, 8, 2, qx, sx, qw, sw, off, dt, y, ws, n, None)

    for kw in (dict(qx=None), dict(sx=None), dict(qw=None), dict(sw=None), dict(off=None),
               dict(dt=3), dict(y=None), dict(qx=FAKE + 8), dict(qw=FAKE + 8), dict(sx=FAKE + 2),
               dict(sw=FAKE + 2), dict(off=FAKE + 2), dict(y=FAKE + 2), dict(y=FAKE + 1, dt=1)):
        assert call(**kw) == 1, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(n=need - 1)):
        assert call(**kw) == 3, kw
    assert call(qx=None, sx=None, y=None, ws=None, n=0, rows=0) == 0


def test_experts_arguments(lib):
    cfg = M.MoeConfig.make(64, 128, 8, 2, 128, n_shared=1)
    need = M.grouped_ffn_int8_workspace_size(cfg)
    m, none = M.MoeInt8Matrix(FAKE, FAKE), M.MoeInt8Matrix()
    good = M.MoeInt8Weights(m, m, m, m, m, m)

    def call(c=cfg, x=FAKE, perm=FAKE, off=FAKE, w=FAKE, wt=good, y=FAKE, ws=FAKE, n=need):
        return lib.moe_grouped_ffn_int8(ctypes.byref(c), x, perm, off, w,
                                        None if wt is None else ctypes.byref(wt), y, ws, n, None)

    for kw in (dict(x=None), dict(perm=None), dict(off=None), dict(wt=None), dict(y=None),
               dict(x=FAKE + 8), dict(y=FAKE + 8), dict(w=FAKE + 2),
               dict(wt=M.MoeInt8Weights(m, none, m, m, m, m)),
               dict(wt=M.MoeInt8Weights(m, m, m, m, m, none)),
               dict(wt=M.MoeInt8Weights(m, m, M.MoeInt8Matrix(FAKE + 4, FAKE), m, m, m))):
        assert call(**kw) == 1, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 64), dict(n=need - 1)):
        assert call(**kw) == 3, kw
    bits = M.MoeConfig.make(64, 128, 8, 2, 128, weight_bits=8)
    assert call(c=bits) == 1
    assert call(c=M.MoeConfig.make(64, 100, 8, 2, 128)) == 2
    empty = M.MoeConfig.make(0, 128, 8, 2, 128)
    assert call(c=empty, x=None, perm=None, off=None, wt=None, y=None, ws=None, n=0) == 0
    assert M.grouped_ffn_int8_workspace_size(empty) == 512
