"""What the check of the few-token layer's waits refuses: on the CPU."""
import ctypes

import pytest

import sparse_moe_layer_route_gb300 as M
from test_few_host import A, B, BASE, OF_EXPERTS, SHAPES, WEIGHTS, OnGpu, calls, lib  # noqa: F401
import torch


@pytest.mark.parametrize("kw,status", [
    (dict(which=-1), 1), (dict(which=3), 1), (dict(limit=99999), 1), (dict(limit=2000000001), 1), (dict(x=None), 1),
    (dict(idx=None), 1), (dict(out=B + 2), 1), (dict(ws=None), 3), (dict(size=512), 3), (dict(T=0), 1), (dict(T=17), 2)])
def test_arguments(lib, kw, status):  # noqa: F811
    v = {**dict(which=0, limit=1000000, x=A, idx=A, out=B, ws=0x100, size=1 << 30, T=4), **kw}
    cfg = M.MoeConfig.make(**{**BASE, "T": v["T"]})
    w = M.make_weights(A, A, A, A, A)
    assert lib.moe_check_few_waits(ctypes.byref(cfg), ctypes.byref(w), v["x"], v["idx"], v["out"], v["ws"], v["size"],
                                   v["which"], v["limit"], None) == status


def call(**change):
    t = {n: OnGpu(torch.zeros(shape, dtype=dtype)) for n, (shape, dtype) in SHAPES.items()}
    t.update(change)
    w = M.make_weights(**{n: t[n] for n in WEIGHTS})
    M.check_few_waits(M.MoeConfig.make(**BASE, n_shared=1), w, t["x"], t["topk_idx"], t["out"], t["ws"], 1, 1000000,
                      stream=0)


@pytest.mark.parametrize("name", [n for n in OF_EXPERTS if n != "topk_w"])
def test_tensors(calls, name):  # noqa: F811
    call()
    assert [c[0] for c in calls] == ["moe_check_few_waits"]
    shape, dtype = SHAPES[name]
    for bad in (OnGpu(torch.zeros(shape, dtype=dtype), 1), torch.zeros(shape, dtype=dtype)):
        with pytest.raises(ValueError):
            call(**{name: bad})
    assert len(calls) == 1
