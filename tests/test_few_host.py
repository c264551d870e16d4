"""What the few-token entry points refuse: on the CPU, by the library itself and by the binding before it."""
import ctypes

import pytest
import torch

import sparse_moe_layer_route_gb300 as M
from sparse_moe_layer_route_gb300 import _build
from test_binding_checks_host import OnGpu, calls  # noqa: F401

BASE = dict(T=4, d=128, E=8, top_k=2, d_ff=64)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return M.lib()


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(T=0), 0), (dict(T=16), 0), (dict(T=17), 2), (dict(T=-1), 1), (dict(E=256, top_k=8), 0),
    (dict(E=257), 2), (dict(d=96), 2), (dict(d=65536, d_ff=65536), 0), (dict(d=65600), 2),
    (dict(d_ff=65600), 2), (dict(weight_bits=8), 2), (dict(overflow_reroute=1), 0),
    (dict(overflow_reroute=1, capacity_override=3), 2), (dict(capacity_factor=1.5), 0),
    (dict(n_groups=4, topk_groups=2), 0), (dict(n_shared=4), 0), (dict(n_shared=5), 2),
    (dict(mode=M.ROUTE_GUMBEL, tau=0.0), 1)])
def test_configurations(lib, kw, status):
    cfg = M.MoeConfig.make(**{**BASE, "d": 128, "d_ff": 128, **kw})
    n = ctypes.c_size_t(0)
    assert lib.moe_few_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == status
    assert n.value >= 512 if status == 0 else n.value == 0
    assert lib.moe_few_workspace_size(ctypes.byref(cfg), None) != 0


def test_a_workspace_serves_fewer_tokens(lib):
    for kw in (BASE, dict(T=1, d=7168, E=128, top_k=2, d_ff=2048, n_shared=1)):
        sizes = [M.few_workspace_size(M.MoeConfig.make(**{**kw, "T": T})) for T in range(17)]
        assert sizes == sorted(sizes)


A, B = 0x10000, 0x20000         # addresses that the library looks at, but never reads: every call is refused


def args(**kw):
    """Arguments of both entry points; none of these calls gets as far as a launch."""
    w = M.make_weights(A, A, A, A, A, A, A, A, W_g_t=A)
    for name in list(kw):
        if hasattr(w, name):
            setattr(w, name, kw.pop(name))
    a = dict(cfg=M.MoeConfig.make(**{**BASE, "n_shared": 1, **kw.pop("cfg", {})}), w=w, x=A, u=A, idx=A,
             gates=A, out=B, ws=0x100, size=1 << 30)
    assert not set(kw) - set(a)
    a.update(kw)
    ref = ctypes.byref
    layer = (ref(a["cfg"]), ref(a["w"]), a["x"], a["u"], a["out"], None, a["ws"], a["size"], None)
    experts = (ref(a["cfg"]), ref(a["w"]), a["x"], a["idx"], a["gates"], a["out"], a["ws"], a["size"],
               None)
    return layer, experts


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(x=A + 8), 1), (dict(out=None), 1), (dict(out=B + 8), 1), (dict(W_gate=None), 1),
    (dict(W_up=None), 1), (dict(W_down=A + 2), 1), (dict(Wsh_gate=None), 1), (dict(Wsh_up=A + 8), 1),
    (dict(Wsh_down=None), 1), (dict(ws=None), 3), (dict(ws=0x180), 3), (dict(size=4096), 3),
    (dict(cfg=dict(T=17)), 2)])
def test_arguments_of_both(lib, kw, status):
    layer, experts = args(**kw)
    assert lib.moe_layer_forward_few(*layer) == status
    assert lib.moe_experts_few(*experts) == status


@pytest.mark.parametrize("kw", [
    dict(W_g=None), dict(W_g_t=A + 8), dict(cfg=dict(mode=M.ROUTE_GUMBEL), u=None),
    dict(cfg=dict(mode=M.ROUTE_GUMBEL), u=A + 2), dict(cfg=dict(mode=M.ROUTE_BIAS_SELECT), expert_bias=None),
    dict(cfg=dict(mode=M.ROUTE_BIAS_SELECT), expert_bias=A + 1)])
def test_arguments_of_the_layer(lib, kw):
    assert lib.moe_layer_forward_few(*args(**kw)[0]) == 1


@pytest.mark.parametrize("kw", [dict(idx=None), dict(idx=A + 2), dict(gates=A + 1)])
def test_arguments_of_the_experts(lib, kw):
    assert lib.moe_experts_few(*args(**kw)[1]) == 1


def test_an_empty_batch_looks_at_nothing(lib):
    layer, experts = args(cfg=dict(T=0), x=None, out=None, ws=None, idx=None)
    assert lib.moe_layer_forward_few(*layer) == 0
    assert lib.moe_experts_few(*experts) == 0


# --------------------------------------------------------------------------------------- the binding
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
SHAPES = {"W_g": ((128, 8), BF16), "expert_bias": ((8,), F32), "W_gate": ((8, 128, 64), BF16),
          "W_up": ((8, 128, 64), BF16), "W_down": ((8, 64, 128), BF16), "Wsh_gate": ((1, 128, 64), BF16),
          "Wsh_up": ((1, 128, 64), BF16), "Wsh_down": ((1, 64, 128), BF16), "W_g_t": ((8, 128), BF16),
          "x": ((4, 128), BF16), "gumbel_u": ((4, 8), F32), "out": ((4, 128), BF16),
          "topk_idx": ((4, 2), I32), "topk_w": ((4, 2), F32), "counts": ((8,), I32),
          "offsets": ((9,), I32), "perm_slot": ((8,), I32), "slot_pos": ((8,), I32),
          "ws": ((8192,), torch.uint8)}
WEIGHTS = tuple(SHAPES)[:9]
ROUTE = ("topk_idx", "topk_w", "counts", "offsets", "perm_slot", "slot_pos")
OF_EXPERTS = tuple(n for n in WEIGHTS if n not in ("W_g", "expert_bias", "W_g_t")) + \
    ("x", "out", "topk_idx", "topk_w", "ws")
OF_LAYER = tuple(SHAPES)


def call(entry, at=0, **change):
    t = {n: OnGpu(torch.zeros(shape, dtype=dtype), at) for n, (shape, dtype) in SHAPES.items()}
    t.update(change)
    cfg = M.MoeConfig.make(**BASE, n_shared=1, mode=M.ROUTE_BIAS_SELECT)
    w = M.make_weights(**{n: t[n] for n in WEIGHTS})
    if entry == "experts_few":
        M.experts_few(cfg, w, t["x"], t["topk_idx"], t["topk_w"], t["out"], t["ws"], stream=0)
    else:
        M.layer_forward_few(cfg, w, t["x"], t["gumbel_u"], t["out"],
                            M.make_route_out(**{n: t[n] for n in ROUTE}), t["ws"], stream=0)


CALLS = [("experts_few", n) for n in OF_EXPERTS] + [("layer_forward_few", n) for n in OF_LAYER]


@pytest.mark.parametrize("entry,name", CALLS)
def test_tensors_that_do_not_fit_are_refused(calls, entry, name):  # noqa: F811
    call(entry)
    assert [c[0] for c in calls] == ["moe_" + entry]
    shape, dtype = SHAPES[name]
    bad = [OnGpu(torch.zeros(shape, dtype=dtype), 1), torch.zeros(shape, dtype=dtype)]
    if name != "ws":                          # whose element type and number do not matter here
        bad += [OnGpu(torch.zeros(*shape[:-1], shape[-1] + 8, dtype=dtype)),
                OnGpu(torch.zeros(shape, dtype=torch.float64)),
                OnGpu(torch.zeros(*shape[:-1], 2 * shape[-1], dtype=dtype)[..., ::2])]
    for t in bad:
        with pytest.raises(ValueError):
            call(entry, **{name: t})
    assert len(calls) == 1


def test_another_gpu_than_the_current_one_is_refused(calls):  # noqa: F811
    for entry in ("experts_few", "layer_forward_few"):
        with pytest.raises(ValueError):
            call(entry, at=1)
    assert calls == []
