"""What the norms around a block and dropout refuse, and the reference's generator: on the CPU."""
import ctypes

import pytest
import torch

import norm_reference as R
import sparse_moe_layer_route_gb300 as M
from sparse_moe_layer_route_gb300 import _build
from test_binding_checks_host import OnGpu, calls  # noqa: F401

F32, BF16, I64 = torch.float32, torch.bfloat16, torch.int64


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return M.lib()


@pytest.mark.parametrize("counter,key,want", [
    # the known answers that its authors published
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_generator(counter, key, want):
    assert R.philox(counter, key) == want


def test_reference_gradient_is_the_forward_pass_s():
    g = torch.Generator().manual_seed(3)
    for after, before in ((1, 1), (2, 2), (0, 1), (1, 0), (0, 2)):
        c = dict(after=after, before=before, alpha=0.8, beta=1.3, eps=1e-5, gate_rows=3)
        T, d = 7, 20
        m = R.factors(1, 2, T, d, 0.3)

        def leaf(*shape):
            return torch.randn(*shape, generator=g).double().requires_grad_(True)

        t = {"h": leaf(T, d), "y": leaf(T, d), "gate": leaf(3, d),
             "w_after": leaf(d) if after else None, "b_after": leaf(d) if after else None,
             "w_before": leaf(d) if before else None, "b_before": leaf(d) if before else None}
        h, n, _, _ = R.forward(c, t, m)
        dh, dn = torch.randn(T, d, generator=g).double(), torch.randn(T, d, generator=g).double()
        loss = (h * dh).sum() + ((n * dn).sum() if before else 0)
        names = [k for k, v in t.items() if v is not None]
        grads = dict(zip(names, torch.autograd.grad(loss, [t[k] for k in names])))
        plain = {k: None if v is None else v.detach() for k, v in t.items()}
        got, _ = R.backward(c, {**plain, "h_out": h.detach(), "d_h_out": dh, "d_n": dn if before else None}, m)
        for k in names:
            assert torch.allclose(got["d_" + k], grads[k], rtol=1e-10, atol=1e-10), k


BASE = dict(T=4, d=96, after=M.NORM_RMS, before=M.NORM_LAYER, gate_rows=2, p_drop=0.1)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(T=0), 0), (dict(T=-1), 1), (dict(d=0), 1), (dict(d=65536), 0), (dict(d=65537), 2),
    (dict(after=3), 1), (dict(before=-1), 1), (dict(h_dtype=3), 1), (dict(y_dtype=-1), 1), (dict(w_dtype=4), 1),
    (dict(gate_rows=-1), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=0.0), 0),
    (dict(alpha=float("inf")), 1), (dict(beta=float("nan")), 1), (dict(p_drop=1.0), 1), (dict(p_drop=-0.1), 1),
    (dict(p_drop=float("nan")), 1), (dict(ld_h=95), 1), (dict(ld_y=95), 1), (dict(ld_h=96, ld_y=200), 0),
    (dict(ld_h=2 ** 61), 2), (dict(ld_y=-5), 1), (dict(T=2 ** 31 - 1), 0)])
def test_configurations(lib, kw, status):
    cfg = M.ResidualNormConfig.make(**{**BASE, **kw})
    n = ctypes.c_size_t(0)
    assert lib.moe_residual_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == status
    assert lib.moe_residual_norm_workspace_size(ctypes.byref(cfg), None) != 0


def test_a_workspace_serves_fewer_tokens(lib):
    sizes = [M.residual_norm_workspace_size(M.ResidualNormConfig.make(T, 512)) for T in
             (0, 1, 2, 3, 100, 319, 320, 321, 5000)]
    assert sizes == sorted(sizes)


A, WS = 0x10000, 0x100             # addresses that are looked at, not read: every call is refused


def forward_args(cfg=None, **kw):
    p = M._NormParams(A, A, A, A, A, A)
    for name, _ in M._NormParams._fields_:
        if name in kw:
            setattr(p, name, kw.pop(name))
    a = dict(h=A, y=A, h_out=A, n=A)
    a.update(kw)
    cfg = M.ResidualNormConfig.make(**{**BASE, **(cfg or {})})
    return cfg, (ctypes.byref(cfg), a["h"], a["y"], ctypes.byref(p), a["h_out"], a["n"], None)


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(h=A + 1), dict(y=None), dict(y=A + 1), dict(h_out=A + 1), dict(n=None), dict(n=A + 1),
    dict(cfg=dict(before=0)), dict(cfg=dict(before=0), n=None), dict(cfg=dict(after=0)), dict(gate=None),
    dict(cfg=dict(gate_rows=0)), dict(rng=None), dict(rng=A + 4), dict(w_after=A + 1), dict(b_before=A + 1),
    dict(cfg=dict(w_dtype=0), gate=A + 2), dict(cfg=dict(h_dtype=0), h=A + 2),
    dict(cfg=dict(before=0), n=None, w_before=None, b_before=None, h_out=None)])
def test_arguments_of_the_forward_pass(lib, kw):
    cfg, args = forward_args(**kw)
    assert lib.moe_residual_norm(*args) == 1


def backward_args(cfg=None, **kw):
    p, g = M._NormParams(A, A, A, A, A, A), M._NormGrads(A, A, A, A, A)
    for name, _ in M._NormParams._fields_:
        if name in kw:
            setattr(p, name, kw.pop(name))
    for name, _ in M._NormGrads._fields_:
        if "d_" + name in kw:
            setattr(g, name, kw.pop("d_" + name))
    a = dict(h_out=A, y=A, d_h_out=A, d_n=A, d_h=A, d_y=A, ws=WS, size=1 << 40)
    assert set(kw) <= set(a), kw
    a.update(kw)
    cfg = M.ResidualNormConfig.make(**{**BASE, **(cfg or {})})
    return (cfg, p, g), (ctypes.byref(cfg), a["h_out"], a["y"], a["d_h_out"], a["d_n"], ctypes.byref(p),
                         a["d_h"], a["d_y"], ctypes.byref(g), a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(h_out=None), 1), (dict(h_out=A + 1), 1), (dict(y=None), 1), (dict(d_y=None), 1), (dict(d_h=None), 1),
    (dict(d_h_out=None, d_n=None), 1), (dict(d_n=A + 1), 1), (dict(d_y=A + 1), 1), (dict(d_h=A + 1), 1),
    (dict(cfg=dict(before=0)), 1), (dict(cfg=dict(before=0), d_w_before=None, d_b_before=None), 1),
    (dict(cfg=dict(after=0), w_after=None, b_after=None), 1), (dict(gate=None), 1),
    (dict(cfg=dict(gate_rows=0), gate=None), 1), (dict(rng=None), 1), (dict(d_w_after=A + 2), 1),
    (dict(ws=None), 3), (dict(ws=WS + 16), 3), (dict(size=9000), 3)])
def test_arguments_of_the_backward_pass(lib, kw, status):
    keep, args = backward_args(**kw)
    assert lib.moe_residual_norm_backward(*args) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(dtype=3), 1), (dict(x=None), 1), (dict(x=A + 1), 1), (dict(y=None), 1),
    (dict(y=A + 1), 1), (dict(r=A + 1), 1), (dict(p=1.0), 1), (dict(p=-0.5), 1), (dict(p=float("nan")), 1),
    (dict(rng=None), 1), (dict(rng=A + 4), 1), (dict(ld_x=95), 1), (dict(ld_r=95), 1), (dict(ld_r=2 ** 61), 2),
    (dict(d=2 ** 31 - 1), 2)])
def test_arguments_of_dropout(lib, kw, status):
    a = dict(T=4, d=96, dtype=1, x=A, ld_x=0, p=0.5, rng=A, r=A, ld_r=0, y=A)
    a.update(kw)
    assert lib.moe_dropout(a["T"], a["d"], a["dtype"], a["x"], a["ld_x"], a["p"], a["rng"], a["r"], a["ld_r"],
                           a["y"], None) == status


# --------------------------------------------------------------------------------------- the binding
T, D = 4, 96
SHAPES = {"h": ((T, D), F32), "y": ((T, D), BF16), "h_out": ((T, D), F32), "n": ((T, D), BF16),
          "w_after": ((D,), BF16), "b_after": ((D,), BF16), "gate": ((2, D), BF16), "w_before": ((D,), BF16),
          "b_before": ((D,), BF16), "rng": ((2,), I64), "d_h_out": ((T, D), F32), "d_n": ((T, D), BF16),
          "d_h": ((T, D), F32), "d_y": ((T, D), BF16), "d_w_after": ((D,), F32), "d_b_after": ((D,), F32),
          "d_gate": ((2, D), F32), "d_w_before": ((D,), F32), "d_b_before": ((D,), F32),
          "ws": ((1 << 16,), torch.uint8), "x": ((T, D), BF16), "residual": ((T, D), BF16),
          "out": ((T, D), BF16)}
FORWARD = ("h", "y", "h_out", "n", "w_after", "b_after", "gate", "w_before", "b_before", "rng")
BACKWARD = ("h_out", "y", "d_h_out", "d_n", "d_h", "d_y", "ws", "w_after", "b_after", "gate", "w_before", "rng",
            "d_w_after", "d_b_after", "d_gate", "d_w_before", "d_b_before")


def call(entry, at=0, **change):
    t = {n: OnGpu(torch.zeros(shape, dtype=dtype), at) for n, (shape, dtype) in SHAPES.items()}
    t.update(change)
    cfg = M.ResidualNormConfig.make(T, D, after=M.NORM_RMS, before=M.NORM_LAYER, h_dtype=M.DTYPE_F32,
                                    gate_rows=3, p_drop=0.1)
    if entry == "dropout":
        M.dropout(t["x"], 0.1, t["rng"], t["out"], residual=t["residual"], stream=0)
    elif entry == "residual_norm":
        M.residual_norm(cfg, *(t[n] for n in FORWARD[:4]), **{n: t[n] for n in FORWARD[4:]}, stream=0)
    else:
        M.residual_norm_backward(cfg, *(t[n] for n in BACKWARD[:7]), **{n: t[n] for n in BACKWARD[7:]}, stream=0)


CALLS = [("residual_norm", n) for n in FORWARD] + [("residual_norm_backward", n) for n in BACKWARD] + \
    [("dropout", n) for n in ("x", "rng", "out", "residual")]


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
    if name in ("x", "residual"):
        bad.append(OnGpu(torch.zeros(1, D, dtype=dtype).expand(T, D)))
    for t in bad:
        with pytest.raises(ValueError):
            call(entry, **{name: t})
    assert len(calls) == 1


def test_another_gpu_than_the_current_one_is_refused(calls):  # noqa: F811
    for entry in ("residual_norm", "residual_norm_backward", "dropout"):
        with pytest.raises(ValueError):
            call(entry, at=1)
    assert calls == []


def test_dropout_takes_rows_of_wider_buffers(calls):  # noqa: F811
    x, r = torch.zeros(T, D + 5, dtype=BF16)[:, :D], torch.zeros(T, 2 * D, dtype=BF16)[:, D:]
    call("dropout", x=OnGpu(x), residual=OnGpu(r))
    (_, args), = calls
    assert args[4] == D + 5 and args[8] == 2 * D
    with pytest.raises(ValueError):
        call("dropout", x=OnGpu(torch.zeros(T, 2, D, dtype=BF16)))
