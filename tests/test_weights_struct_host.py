"""make_weights and make_route_out hold the tensors they were made of, which the few-token entry points check; an address
that the program sets itself is its own affair, and the tensor it replaces is let go."""
import gc
import weakref

import pytest
import torch

import sparse_moe_layer_route_gb300 as M
from test_few_host import BASE, ROUTE, SHAPES, WEIGHTS, OnGpu, calls  # noqa: F401


def tensors(**change):
    t = {n: OnGpu(torch.zeros(shape, dtype=dtype)) for n, (shape, dtype) in SHAPES.items()}
    return {**t, **change}


def run(t, w, r):
    M.layer_forward_few(M.MoeConfig.make(**BASE, n_shared=1, mode=M.ROUTE_BIAS_SELECT), w, t["x"], None, t["out"], r,
                        t["ws"], stream=0)


@pytest.mark.parametrize("name", WEIGHTS)
def test_an_address_set_anew_is_not_checked_as_the_old_tensor(calls, name):  # noqa: F811
    t = tensors(**{name: OnGpu(torch.zeros(3, 5))})
    w, r = M.make_weights(**{n: t[n] for n in WEIGHTS}), M.make_route_out(**{n: t[n] for n in ROUTE})
    with pytest.raises(ValueError):
        run(t, w, r)
    setattr(w, name, 4096)
    run(t, w, r)
    (_, args), = calls
    assert getattr(args[1]._obj, name) == 4096


@pytest.mark.parametrize("name", ROUTE)
def test_results_set_anew(calls, name):  # noqa: F811
    t = tensors(**{name: OnGpu(torch.zeros(3, 5))})
    w, r = M.make_weights(**{n: t[n] for n in WEIGHTS}), M.make_route_out(**{n: t[n] for n in ROUTE})
    with pytest.raises(ValueError):
        run(t, w, r)
    setattr(r, name, None)
    run(t, w, r)
    assert len(calls) == 1


def test_what_is_held_and_let_go():
    t = [torch.zeros(4, 4) for _ in range(6)]
    seen = [weakref.ref(v) for v in t]
    w, r = M.make_weights(*t[:5]), M.make_route_out(topk_w=t[5])
    del t
    gc.collect()
    assert all(v() is not None for v in seen)
    w.W_gate = 4096
    r.topk_w = None
    gc.collect()
    assert [v() is None for v in seen] == [False, False, True, False, False, True]
    del w
    gc.collect()
    assert all(v() is None for v in seen)
